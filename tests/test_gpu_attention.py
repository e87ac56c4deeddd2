"""The attention operators on the GPU against the float64 oracle.

Tolerances, per element, with u = half a step of the output type, e = 2^-24:
  norm + rotation   10 float32 roundings on the way (mean of D squares: D e more,
                    halved by the root), then one to the output type;
  attention         a score is off by at most (D + 4) e sum|q k| scale, so a
                    probability by twice that (its own and the sum's) relative,
                    plus the exponential's 2^-22 and n e of the sums; probabilities
                    are rounded to the type before they meet V (u again);
  backward          the same through P, dP = dO V^T and delta = rowsum(dO O), the
                    rounding of P and dS to the type, and one of the result.
Each bound is a sum of absolute terms formed in float64 beside the result."""
import numpy as np
import pytest

from oracle import attention as A

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -150}   # half the smallest subnormal step


def f8(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, tol, what=""):
    got, ref = f8(got), np.asarray(ref)
    assert got.shape == ref.shape
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    bad = off > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(off / np.maximum(tol, 1e-300)):.2f} x the bound"


def normal(seed, *shape, dtype="float32", scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(getattr(torch, dtype)).cuda()


def ok(bl):
    assert bl.sync_status() == "BL_OK"


# ---- norms and rotation ---------------------------------------------------------------------------------------------

def rows(seed, m, hq, hk, d, rot, dtype="float32"):
    import torch
    qkv = normal(seed, m, (hq + 2 * hk) * d)
    qkv *= torch.logspace(-2, 2, m, device="cuda")[:, None] if m else 1
    pos = torch.from_numpy(np.random.default_rng(seed).integers(0, 5000, m).astype(np.int32)).cuda()
    return qkv, pos, 1 + 0.3 * normal(seed + 1, d), 1 + 0.3 * normal(seed + 2, d)


def split(x, hq, hk, d):
    m = x.shape[0]
    return [y.reshape(m, -1, d) for y in np.split(x, [hq * d, (hq + hk) * d], 1)]


SHAPES = [(1, 20, 5, 128, 128, False, "bfloat16"), (7, 4, 4, 32, 16, True, "float32"), (33, 6, 2, 80, 80, False, "float16"),
          (3, 3, 1, 8, 8, True, "bfloat16"), (5, 2, 2, 256, 64, False, "float32"), (300, 32, 8, 128, 128, True, "float16"),
          (4, 5, 1, 96, 0, False, "float32"), (2, 1, 1, 24, 8, False, "float16"), (900, 8, 8, 64, 64, False, "bfloat16"),
          # enough rows for the kernels that are fed by bulk copies, each number of lanes a head
          (4801, 12, 4, 32, 32, False, "float16"), (2401, 20, 5, 56, 24, True, "float32"),
          (1705, 20, 4, 128, 128, False, "bfloat16"), (1301, 18, 9, 256, 64, True, "float32"),
          (4803, 2, 1, 80, 40, False, "bfloat16"), (4802, 1, 1, 8, 8, False, "float32")]


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dtype", SHAPES)
def test_norm_rope(bl, m, hq, hk, d, rot, inter, dtype):
    import torch
    qkv, pos, gq, gk = rows(m + d, m, hq, hk, d, rot)
    table = bl.rope_table(5000, rot) if rot else None
    t = None if table is None else table.cpu().numpy()
    got = bl.qk_norm_rope(qkv, hq, hk, d, pos, table, gq, gk, eps=1e-5, dtype=getattr(torch, dtype), interleaved=inter)
    ok(bl)
    q, k, v = split(f8(qkv), hq, hk, d)
    for x, y, g in ((q, got[0], gq), (k, got[1], gk)):
        ref = A.norm_rope(x, pos.cpu().numpy(), t, f8(g), 1e-5, inter)
        y0 = A.norm_rope(x, pos.cpu().numpy(), None, f8(g), 1e-5)
        a, b = A.rotation_pairs(rot, inter)
        size = np.abs(y0)
        size[..., a], size[..., b] = [np.hypot(y0[..., a], y0[..., b])] * 2
        within(y, ref, HALF[dtype] * np.abs(ref) + (10 + d / 2) * E * size * 1.5 + TINY[dtype], "q or k")
    within(got[2], v, HALF[dtype] * np.abs(v) + TINY[dtype], "v")


def test_rope_table(bl):
    for p, r, base in ((1, 2, 1e4), (777, 80, 5e5), (131072, 8, 1e4)):
        got, ref = bl.rope_table(p, r, base).cpu().numpy(), A.rope_table(p, r, base)
        # the angle in float64: 2^-52 relative of up to p, then one rounding of the cosine
        assert np.abs(got.astype(np.float64) - ref.astype(np.float64)).max() <= 2 * E + p * 2.0 ** -50


def test_norm_rope_separate_rows_with_strides(bl):
    import torch
    m, hq, hk, d = 9, 4, 2, 64
    wide = normal(4, m, 3, 512)
    parts = (wide[:, 0, :hq * d], wide[:, 1, 16:16 + hk * d], wide[:, 2, 100:100 + hk * d])
    pos = torch.arange(m, dtype=torch.int32, device="cuda")
    table = bl.rope_table(m, d)
    got = bl.qk_norm_rope(parts, hq, hk, d, pos, table, dtype=torch.float32)
    ref = bl.qk_norm_rope(torch.cat(parts, 1).contiguous(), hq, hk, d, pos, table, dtype=torch.float32)
    ok(bl)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    with pytest.raises(bl.BitLinearError, match="ALIGNMENT"):
        bl.qk_norm_rope((parts[0], wide[:, 1, 17:17 + hk * d], parts[2]), hq, hk, d, pos, table)


@pytest.mark.parametrize("page", [1, 16, 24])
def test_append_fills_only_its_slots(bl, page):
    import torch
    m, hq, hk, d = 37, 8, 2, 128
    qkv, pos, gq, gk = rows(page, m, hq, hk, d, d)
    table = bl.rope_table(5000, d)
    n = -(-2 * m // page) + 1
    kc, vc = normal(1, n, hk, page, d, dtype="bfloat16"), normal(2, n, hk, page, d, dtype="bfloat16")
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.from_numpy(np.random.default_rng(page).permutation(n * page)[:m]).cuda()
    slots[5] = -1
    q = bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, kc, vc, slots)
    rq, rk, rv = bl.qk_norm_rope(qkv, hq, hk, d, pos, table, gq, gk)
    ok(bl)
    assert torch.equal(q, rq)
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            k0[s // page, :, s % page], v0[s // page, :, s % page] = rk[i], rv[i]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_of_many_rows(bl):
    """As many rows as the kernel fed by bulk copies takes, some without a slot, some out of range."""
    import torch
    m, hq, hk, d, page = 2400, 12, 2, 64, 16
    qkv, pos, gq, gk = rows(3, m, hq, hk, d, d)
    table = bl.rope_table(5000, d)
    n = m // page + 7
    kc, vc = torch.zeros(n, hk, page, d, dtype=torch.float16, device="cuda"), torch.zeros(n, hk, page, d, dtype=torch.float16, device="cuda")
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.from_numpy(np.random.default_rng(1).permutation(n * page)[:m]).cuda()
    slots[7::100] = -1
    q = bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, kc, vc, slots)
    rq, rk, rv = bl.qk_norm_rope(qkv, hq, hk, d, pos, table, gq, gk, dtype=torch.float16)
    ok(bl)
    keep = slots >= 0
    k0[slots[keep] // page, :, slots[keep] % page], v0[slots[keep] // page, :, slots[keep] % page] = rk[keep], rv[keep]
    assert torch.equal(q, rq) and torch.equal(kc, k0) and torch.equal(vc, v0)
    pos[11], slots[13] = 5000, n * page
    before = kc.clone()
    bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, kc, vc, slots)
    assert bl.sync_status() == "BL_ERR_RANGE"
    assert torch.equal(kc, before)


def test_bad_positions_and_slots_are_reported_and_not_written(bl):
    import torch
    m, hq, hk, d = 6, 2, 1, 32
    qkv, pos, gq, gk = rows(8, m, hq, hk, d, d)
    table = bl.rope_table(100, d)
    pos = torch.tensor([0, -1, 99, 100, 5, 6], dtype=torch.int32, device="cuda")
    kc, vc = torch.zeros(2, hk, 4, d, dtype=torch.float16, device="cuda"), torch.zeros(2, hk, 4, d, dtype=torch.float16, device="cuda")
    slots = torch.tensor([0, 1, 2, 3, 8, 1 << 40], device="cuda")
    bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, kc, vc, slots)
    assert bl.sync_status() == "BL_ERR_RANGE"
    ok(bl)
    held = kc.abs().sum((1, 3)).flatten().tolist()
    assert [x > 0 for x in held] == [True, False, True, False] + [False] * 4


def test_norm_rope_reports_nonfinite(bl):
    import torch
    qkv, pos, gq, gk = rows(8, 4, 2, 1, 32, 32)
    table = bl.rope_table(5000, 32)
    clean = bl.qk_norm_rope(qkv, 2, 1, 32, pos, table, gq, gk)
    for col in (3, 70, 100):
        x = qkv.clone()
        x[2, col] = float("inf") if col == 70 else float("nan")
        got = bl.qk_norm_rope(x, 2, 1, 32, pos, table, gq, gk)
        assert bl.sync_status() == "BL_ERR_NONFINITE"
        for a, b in zip(got, clean):
            assert torch.equal(a[[0, 1, 3]], b[[0, 1, 3]])


@pytest.mark.parametrize("m", [3, 5000])
def test_large_values_are_no_error(bl, m):
    """A value's square may overflow float32: values are only converted."""
    import torch
    qkv, pos, gq, gk = rows(8, m, 2, 1, 32, 32)
    qkv[1, 96:] = 1e25
    table = bl.rope_table(5000, 32)
    v = bl.qk_norm_rope(qkv, 2, 1, 32, pos, table, gq, gk)[2]
    ok(bl)
    assert torch.equal(v[1, 0], qkv[1, 96:].bfloat16())
    qkv[1, 100] = float("-inf")
    bl.qk_norm_rope(qkv, 2, 1, 32, pos, table, gq, gk)
    assert bl.sync_status() == "BL_ERR_NONFINITE"


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dtype", SHAPES)
def test_norm_rope_backward(bl, m, hq, hk, d, rot, inter, dtype):
    qkv, pos, gq, gk = rows(m + d, m, hq, hk, d, rot)
    table = bl.rope_table(5000, rot) if rot else None
    t = None if table is None else table.cpu().numpy()
    dq, dk, dv = (normal(n, m, h, d, dtype=dtype) for n, h in ((3, hq), (4, hk), (5, hk)))
    dx, dgq, dgk = bl.qk_norm_rope_backward(dq, dk, dv, qkv, hq, hk, d, pos, table, gq, gk, eps=1e-5, interleaved=inter)
    ok(bl)
    q, k, _ = split(f8(qkv), hq, hk, d)
    p = pos.cpu().numpy()
    gots = split(f8(dx), hq, hk, d)
    for x, dz, got, g, dg in ((q, dq, gots[0], gq, dgq), (k, dk, gots[1], gk, dgk)):
        rx, rg = A.norm_rope_backward(f8(dz), x, p, t, f8(g), 1e-5, inter)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        dy = np.abs(f8(dz))
        a, b = A.rotation_pairs(rot, inter)
        dy[..., a], dy[..., b] = [np.abs(f8(dz))[..., a] + np.abs(f8(dz))[..., b]] * 2
        gy, xr = dy * np.abs(f8(g)), np.abs(x * r)
        size = r * (gy + xr * (xr * gy).mean(-1, keepdims=True))
        assert (np.abs(got - rx) <= (20 + 2 * d) * E * size).all()
        terms = (dy * xr).sum((0, 1))
        within(dg, rg, (16 + d + m * x.shape[1]) * E * terms, "dg")
    assert np.array_equal(gots[2], f8(dv))


def test_norm_rope_backward_repeats_bit_for_bit(bl):
    import torch
    qkv, pos, gq, gk = rows(2, 700, 8, 2, 64, 64)
    table = bl.rope_table(5000, 64)
    dq, dk, dv = (normal(n, 700, h, 64) for n, h in ((3, 8), (4, 2), (5, 2)))
    one, two = (bl.qk_norm_rope_backward(dq, dk, dv, qkv, 8, 2, 64, pos, table, gq, gk) for _ in range(2))
    for a, b in zip(one, two):
        assert torch.equal(a, b)


def test_no_rows(bl):
    import torch
    qkv, table = torch.empty(0, 6 * 32, device="cuda"), bl.rope_table(10, 32)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    q, k, v = bl.qk_norm_rope(qkv, 4, 1, 32, pos, table)
    assert q.shape == (0, 4, 32)
    dx, dgq, dgk = bl.qk_norm_rope_backward(q, k, v, qkv, 4, 1, 32, pos, table)
    assert dx.shape == (0, 192) and not dgq.any() and not dgk.any()
    ok(bl)


# ---- attention over packed sequences ----------------------------------------------------------------------------------

def packed(seed, lq, lk, hq, hk, d, dtype, scale=1.0):
    import torch
    cu = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")  # noqa: E731
    return (normal(seed, sum(lq), hq, d, dtype=dtype, scale=scale), normal(seed + 1, sum(lk), hk, d, dtype=dtype),
            normal(seed + 2, sum(lk), hk, d, dtype=dtype), cu(lq), cu(lk))


def score_slack(q, k, d):
    """Relative error of a probability: twice the score's, plus the exponential's."""
    qk = np.einsum("ihd,jhd->hij", np.abs(q), np.repeat(np.abs(k), q.shape[1] // k.shape[1], 1)).max(initial=0.0)
    return 2 * (d + 4) * E * qk / np.sqrt(d) + 2.0 ** -21


def check_forward(q, k, v, cq, ck, window, sinks, out, lse, dtype):
    cq, ck = cq.tolist(), ck.tolist()
    q, k, v = f8(q), f8(k), f8(v)
    out, lse = f8(out), f8(lse)
    d, group = q.shape[2], q.shape[1] // k.shape[1]
    for b in range(len(cq) - 1):
        i, j = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        ro, rl, p = A.attention(q[i], k[j], v[j], window, sinks)
        see = A.visible(ro.shape[0], k[j].shape[0], window, sinks)
        slack = score_slack(q[i], np.where(see.any(0)[:, None, None], k[j], 0), d) + (k[j].shape[0] + 8) * E
        vv = np.where(see.any(0)[:, None, None], np.abs(v[j]), 0)
        size = np.einsum("hij,jhd->ihd", p, np.repeat(vv, group, 1))
        top = vv.max(initial=0.0)
        tol = HALF[dtype] * (np.abs(ro) + size) + slack * size + TINY[dtype] + k[j].shape[0] * 2.0 ** -31 * top
        assert np.isfinite(out[i]).all()
        off = np.abs(out[i] - ro)
        assert (off <= tol).all(), f"sequence {b}: worst {np.max(off / np.maximum(tol, 1e-300)):.2f} x the bound"
        some = np.isfinite(rl)
        assert np.array_equal(some, np.isfinite(lse[:, i]))
        assert (lse[:, i][~some] == -np.inf).all() and not out[i][~see.any(1)].any()
        assert (np.abs(lse[:, i][some] - rl[some]) <= slack + 4 * E * np.abs(rl[some])).all()


CASES = [  # query lengths, key lengths (None: the same), heads, kv heads, D, window, sinks, type
    ([1], None, 1, 1, 64, 0, 0, "bfloat16"),
    ([128], None, 2, 1, 128, 0, 0, "bfloat16"),
    ([129, 1, 127, 300], None, 4, 4, 32, 0, 0, "float16"),
    ([257, 40], None, 6, 2, 80, 100, 3, "float16"),
    ([64, 500], [200, 777], 4, 1, 128, 0, 0, "bfloat16"),
    ([333], [700], 5, 5, 64, 130, 4, "bfloat16"),
    ([1, 1, 1], [300, 1, 128], 8, 2, 128, 0, 0, "float16"),
    ([300], [100], 2, 2, 64, 0, 0, "bfloat16"),             # more queries than keys: rows that see nothing
    ([0, 50, 0, 70], [30, 50, 0, 70], 2, 1, 96, 0, 0, "float16"),
    ([40, 3], [0, 3], 2, 1, 64, 0, 0, "bfloat16"),          # a sequence without keys
    ([400], None, 2, 1, 64, 1, 0, "bfloat16"),              # a window of one
    ([600], None, 3, 1, 128, 37, 200, "bfloat16"),          # sinks wider than a tile
    ([513], None, 1, 1, 8, 0, 0, "float16"),
    ([700], None, 2, 2, 128, 300, 1, "float16"),
    ([300], None, 16, 1, 64, 64, 0, "bfloat16"),
    ([150], None, 2, 1, 64, 1 << 30, 5, "float16"),         # a window wider than any sequence
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,window,sinks,dtype", CASES)
def test_attention(bl, lq, lk, hq, hk, d, window, sinks, dtype):
    q, k, v, cq, ck = packed(sum(lq) + d, lq, lk or lq, hq, hk, d, dtype)
    out, lse = bl.attention(q, k, v, cq, ck, max(lq), window=window, sinks=sinks)
    ok(bl)
    check_forward(q, k, v, cq, ck, window, sinks, out, lse, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_attention_with_peaked_scores(bl, dtype):
    """Scores far apart (scale 12): running maxima rise many times along a row."""
    q, k, v, cq, ck = packed(3, [390], [390], 4, 2, 64, dtype, scale=12.0)
    k[200:260] *= 3
    out, lse = bl.attention(q, k, v, cq, ck, 390)
    ok(bl)
    check_forward(q, k, v, cq, ck, 0, 0, out, lse, dtype)


def test_attention_strided_rows_scale_and_rows_behind(bl):
    """q, k, v as columns of one buffer; rows behind the last sequence keep what they held."""
    import torch
    n, hq, hk, d = 200, 4, 2, 64
    buf = normal(5, n + 9, (hq + 2 * hk) * d, dtype="bfloat16")
    q = buf[:, :hq * d].unflatten(1, (hq, d))
    k = buf[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    v = buf[:, (hq + hk) * d:].unflatten(1, (hk, d))
    buf[n:] = float("nan")
    cu = torch.tensor([0, 77, n], dtype=torch.int32, device="cuda")
    out = torch.full((n + 9, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, n + 9), 7.0, device="cuda")
    bl.attention(q, k, v, cu, cu, 123, scale=0.3, out=out, lse=lse)
    ref, rl = bl.attention((q[:n].float() * (0.3 * 8)).bfloat16().contiguous(), k[:n].contiguous(), v[:n].contiguous(), cu, cu, 123)
    ok(bl)
    assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()
    assert (out[:n].float() - ref.float()).abs().max() < 0.2          # q rounded again: a loose look
    q8, k8, v8 = (f8(t[:n]) for t in (q, k, v))
    ro, _, p = A.attention(q8[:77], k8[:77], v8[:77], scale=0.3)
    size = np.einsum("hij,jhd->ihd", p, np.repeat(np.abs(v8[:77]), 2, 1))
    within(out[:77], ro, HALF["bfloat16"] * (np.abs(ro) + size) + (3 * score_slack(q8[:77], k8[:77], d) + 99 * E) * size)


def test_masked_places_may_hold_anything(bl):
    """NaN and infinities in keys and values that no row sees: other sequences' padding, beyond the window."""
    import torch
    q, k, v, cq, ck = packed(6, [100, 90], [400, 90], 2, 1, 64, "bfloat16")
    want = bl.attention(q, k, v, cq, ck, 100, window=50, sinks=2)
    for t in (k, v):
        t[2:300 - 49] = float("nan")                       # outside every window, past the sinks
    got = bl.attention(q, k, v, cq, ck, 100, window=50, sinks=2)
    ok(bl)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the next sequence is all NaN: the first one's rows stay what they were, and the status says so
    k[400:], v[400:] = float("nan"), float("inf")
    got = bl.attention(q, k, v, cq, ck, 100, window=50, sinks=2)
    assert bl.sync_status() == "BL_ERR_NONFINITE"
    assert torch.equal(got[0][:100], want[0][:100])


def test_bad_bounds_are_reported(bl):
    import torch
    q, k, v, cq, ck = packed(6, [50, 60, 40], [50, 60, 40], 2, 1, 64, "bfloat16")
    want, _ = bl.attention(q, k, v, cq, ck, 60)
    ok(bl)
    out = torch.full_like(want, 3.0)
    bl.attention(q, k, v, cq, ck, 55, out=out)             # the second is longer than max_q
    assert bl.sync_status() == "BL_ERR_RANGE"
    assert torch.equal(out[:50], want[:50]) and (out[50:110] == 3).all() and torch.equal(out[110:], want[110:])
    bad = torch.tensor([0, 50, 40, 999999], dtype=torch.int32, device="cuda")
    out = torch.full_like(want, 3.0)
    bl.attention(q, k, v, bad, ck, 60, out=out)
    assert bl.sync_status() == "BL_ERR_RANGE"
    assert torch.equal(out[:50], want[:50]) and (out[50:] == 3).all()


def test_nothing_but_empty_sequences(bl):
    import torch
    q, k, v, _, _ = packed(6, [5], [7], 2, 1, 64, "float16")
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 2.0), torch.full((2, 5), 3.0, device="cuda")
    bl.attention(q, k, v, zero, zero, 0, out=out, lse=lse)
    grads = tuple(torch.full_like(t, 4.0) for t in (q, k, k))
    bl.attention_backward(q, q, k, v, out, lse, zero, zero, 0, 0, grads=grads)
    ok(bl)
    assert (out == 2).all() and (lse == 3).all() and all((g == 4).all() for g in grads)
    # keys without queries: their gradients are zero
    cq, ck = zero[:2].contiguous(), torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    empty = q[:0].contiguous()
    o, l = bl.attention(empty, k, v, cq, ck, 0)
    dq, dk, dv = bl.attention_backward(o, empty, k, v, o, l, cq, ck, 0, 7)
    ok(bl)
    assert o.shape == (0, 2, 64) and dq.shape == o.shape and not dk.any() and not dv.any()


def check_backward(q, k, v, cq, ck, window, sinks, out, lse, dout, grads, dtype):
    cq, ck = cq.tolist(), ck.tolist()
    q, k, v, out, lse, dout = (f8(t) for t in (q, k, v, out, lse, dout))
    grads = [f8(t) for t in grads]
    d, hq, group = q.shape[2], q.shape[1], q.shape[1] // k.shape[1]
    u, scale = HALF[dtype], 1 / np.sqrt(d)
    for b in range(len(cq) - 1):
        i, j = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        nk, nq = ck[b + 1] - ck[b], cq[b + 1] - cq[b]
        ref = A.attention_backward(dout[i], q[i], k[j], v[j], out[i], lse[:, i], window, sinks)
        see = A.visible(nq, nk, window, sinks)
        rel = score_slack(q[i], k[j], d) + 2 * E * np.abs(np.where(np.isfinite(lse[:, i]), lse[:, i], 0)).max(initial=0.0)
        size = [np.zeros_like(r) for r in ref]
        for h in range(hq):
            g = h // group
            low = np.where(np.isfinite(lse[h, i]), lse[h, i], 0)[:, None]
            p = np.where(see, np.exp(np.where(see, q[i, h] @ k[j, g].T * scale, 0) - low), 0)
            dp, delta = dout[i, h] @ v[j, g].T, (dout[i, h] * out[i, h]).sum(1, keepdims=True)
            dpa = np.abs(dout[i, h]) @ np.abs(v[j, g]).T + (np.abs(dout[i, h]) * np.abs(out[i, h])).sum(1, keepdims=True)
            ds = np.abs(p * (dp - delta)) * (u + rel) + p * dpa * (d + 4) * E
            if dtype == "float16":                         # P and dS are scaled to keep their last bits
                ds = ds + dpa.max(initial=0.0) * 2.0 ** -36
            more = (nq + nk) * E
            size[0][:, h] += scale * (ds + more * np.abs(p * (dp - delta))) @ np.abs(k[j, g])
            size[1][:, g] += scale * (ds + more * np.abs(p * (dp - delta))).T @ np.abs(q[i, h])
            size[2][:, g] += (p * (u + rel + more * group) + 2.0 ** -36).T @ np.abs(dout[i, h])
        for n, (got, s) in enumerate(zip(grads, (i, j, j))):
            tol = u * np.abs(ref[n]) + size[n] + TINY[dtype]
            off = np.abs(got[s] - ref[n])
            assert np.isfinite(got[s]).all()
            assert (off <= tol).all(), f"sequence {b}, {'qkv'[n]}: worst {np.max(off / np.maximum(tol, 1e-300)):.2f} x the bound"


@pytest.mark.parametrize("lq,lk,hq,hk,d,window,sinks,dtype", CASES)
def test_attention_backward(bl, lq, lk, hq, hk, d, window, sinks, dtype):
    lk = lk or lq
    q, k, v, cq, ck = packed(sum(lq) + d, lq, lk, hq, hk, d, dtype)
    out, lse = bl.attention(q, k, v, cq, ck, max(lq), window=window, sinks=sinks)
    dout = normal(99, *q.shape, dtype=dtype)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, max(lq), max(lk), window=window, sinks=sinks)
    ok(bl)
    check_backward(q, k, v, cq, ck, window, sinks, out, lse, dout, grads, dtype)


@pytest.mark.parametrize("dtype,size", [("float16", 1e-4), ("float16", 100.0), ("bfloat16", 1e-6)])
def test_attention_backward_of_small_and_large_gradients(bl, dtype, size):
    import torch
    q, k, v, cq, ck = packed(5, [300], [300], 2, 1, 64, dtype)
    out, lse = bl.attention(q, k, v, cq, ck, 300)
    one = normal(98, *q.shape, dtype="float32")
    dout = (one * size).to(q.dtype)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, 300, 300)
    ok(bl)
    check_backward(q, k, v, cq, ck, 0, 0, out, lse, dout, grads, dtype)


def test_attention_backward_repeats_and_leaves_other_rows(bl):
    import torch
    q, k, v, cq, ck = packed(11, [200, 190, 9], [260, 190, 9], 4, 1, 64, "bfloat16")
    cq, ck = cq[:3].contiguous(), ck[:3].contiguous()       # the third sequence's rows belong to none
    out, lse = bl.attention(q, k, v, cq, ck, 200)
    dout = normal(97, *q.shape, dtype="bfloat16")
    for t in (q, k, v, dout, out):
        t[-9:] = float("nan")
    runs = []
    for _ in range(2):
        grads = tuple(torch.full_like(t, 5.0) for t in (q, k, k))
        runs.append(bl.attention_backward(dout, q, k, v, out, lse, cq, ck, 200, 260, grads=grads))
    ok(bl)
    for a, b in zip(*runs):
        assert torch.equal(a, b)
        assert (a[-9:] == 5).all() and not (a[:-9] == 5).all()


# ---- paged -----------------------------------------------------------------------------------------------------------

def paged(seed, lens, hq, hk, d, page, dtype):
    import torch
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    at = rng.permutation(total)
    pages = rng.integers(-5, 10 ** 6, (len(lens), max(need + [1]))).astype(np.int32)    # unused entries: anything
    used = 0
    kc, vc = (torch.full((total, hk, page, d), float("nan"), dtype=getattr(torch, dtype), device="cuda") for _ in range(2))
    for b, n in enumerate(need):
        pages[b, :n] = at[used:used + n]
        used += n
    q = normal(seed, len(lens), hq, d, dtype=dtype)
    k, v = normal(seed + 1, sum(lens), hk, d, dtype=dtype), normal(seed + 2, sum(lens), hk, d, dtype=dtype)
    row = 0
    for b, n in enumerate(lens):                            # what no token fills stays NaN
        for j in range(0, n, page):
            m = min(page, n - j)
            kc[pages[b, j // page], :, :m] = k[row + j:row + j + m].transpose(0, 1)
            vc[pages[b, j // page], :, :m] = v[row + j:row + j + m].transpose(0, 1)
        row += n
    return q, kc, vc, torch.from_numpy(pages).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), f8(k), f8(v)


def check_paged(q, k, v, lens, window, sinks, got, dtype):
    q, out, row = f8(q), f8(got), 0
    d, group = q.shape[2], q.shape[1] // k.shape[1]
    for b, n in enumerate(lens):
        kk, vv = k[row:row + n], v[row:row + n]
        row += n
        ro, _, p = A.attention(q[b:b + 1], kk, vv, window, sinks)
        size = np.einsum("hij,jhd->ihd", p, np.repeat(np.abs(vv), group, 1))[0]
        slack = score_slack(q[b:b + 1], kk, d) + (n + 40) * E
        tol = HALF[dtype] * np.abs(ro[0]) + slack * size + TINY[dtype]
        off = np.abs(out[b] - ro[0])
        assert np.isfinite(out[b]).all() and (off <= tol).all(), \
            f"sequence {b} ({n} tokens): worst {np.max(off / np.maximum(tol, 1e-300)):.2f} x the bound"


PAGED = [([1], 1, 1, 64, 16, 0, 0, "bfloat16", "float32"), ([301], 20, 5, 128, 16, 0, 0, "bfloat16", "float32"),
         ([64, 65, 63, 1, 128], 4, 4, 32, 1, 0, 0, "float16", "float16"),
         ([500, 3, 0, 900, 1], 8, 2, 80, 24, 0, 0, "float16", "float32"),
         ([2000, 1500], 32, 8, 128, 64, 0, 0, "bfloat16", "bfloat16"),
         ([700, 90, 650], 6, 2, 64, 16, 100, 4, "bfloat16", "float32"),
         ([1000], 4, 1, 128, 16, 1, 0, "float16", "float32"),
         ([1000, 77], 4, 1, 96, 48, 64, 200, "bfloat16", "float32"),
         ([333, 100], 12, 1, 128, 16, 0, 0, "bfloat16", "float32"),     # 12 heads share a key head
         ([400] * 3, 40, 1, 64, 128, 50, 1, "float16", "float16"),      # 40 of them: several chunks
         ([129], 3, 3, 8, 7, 0, 0, "bfloat16", "float32"),
         ([7, 0, 300] * 70, 2, 1, 32, 16, 0, 0, "float16", "float32")]


@pytest.mark.parametrize("lens,hq,hk,d,page,window,sinks,dtype,out", PAGED)
def test_paged_attention(bl, lens, hq, hk, d, page, window, sinks, dtype, out):
    import torch
    q, kc, vc, pages, n, k, v = paged(len(lens) + d, lens, hq, hk, d, page, dtype)
    ws = bl.workspace(bl.paged_attention_workspace_size(len(lens), hq, kc), "cuda")
    got = [bl.paged_attention(q, kc, vc, pages, n, window=window, sinks=sinks, out_dtype=getattr(torch, out), ws=ws)
           for _ in range(2)]
    ok(bl)
    assert torch.equal(got[0], got[1])                                   # fixed order, counters left at zero
    assert not ws[:2048].any()
    check_paged(q, k, v, lens, window, sinks, got[0], out)


def test_paged_attention_of_one_long_sequence_in_float16_pages(bl):
    import torch
    lens = [40_001, 9]
    q, kc, vc, pages, n, k, v = paged(4, lens, 4, 1, 64, 64, "float16")
    got = bl.paged_attention(q, kc, vc, pages, n)
    ok(bl)
    check_paged(q, k, v, lens, 0, 0, got, "float32")


def test_paged_pages_past_32_bit_offsets(bl):
    """A cache of more than 2^31 elements: pages at its far end."""
    import torch
    hk, page, d = 8, 128, 128
    total = (1 << 31) // (hk * page * d) + 40
    kc = torch.zeros(total, hk, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k, v = normal(1, 300, hk, d, dtype="bfloat16"), normal(2, 300, hk, d, dtype="bfloat16")
    q = normal(3, 1, 8, d, dtype="bfloat16")
    at = [total - 1, total - 30, total - 7]
    for i, p in enumerate(at):
        m = min(page, 300 - i * page)
        kc[p, :, :m], vc[p, :, :m] = (t[i * page:i * page + m].transpose(0, 1) for t in (k, v))
    got = bl.paged_attention(q, kc, vc, torch.tensor([at], dtype=torch.int32, device="cuda"),
                             torch.tensor([300], dtype=torch.int32, device="cuda"))
    ok(bl)
    check_paged(q, f8(k), f8(v), [300], 0, 0, got, "float32")
    del kc, vc
    torch.cuda.empty_cache()


def test_paged_bad_pages_and_lengths(bl):
    import torch
    lens = [100, 50, 60]
    q, kc, vc, pages, n, k, v = paged(4, lens, 4, 2, 64, 16, "bfloat16")
    want = bl.paged_attention(q, kc, vc, pages, n)
    ok(bl)
    pages[1, 2] = kc.shape[0]
    pages[1, 1] = -1
    got = bl.paged_attention(q, kc, vc, pages, n)
    assert bl.sync_status() == "BL_ERR_RANGE"
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and torch.isfinite(got).all()
    n[1] = -3
    got = bl.paged_attention(q, kc, vc, pages, n)
    assert bl.sync_status() == "BL_ERR_RANGE"
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and not got[1].any()


def test_paged_nonfinite_key_is_reported_and_stays_in_its_sequence(bl):
    import torch
    lens = [100, 200]
    q, kc, vc, pages, n, k, v = paged(4, lens, 4, 2, 64, 16, "bfloat16")
    want = bl.paged_attention(q, kc, vc, pages, n)
    ok(bl)
    vc[pages[1, 3], 0, 5] = float("nan")
    got = bl.paged_attention(q, kc, vc, pages, n)
    assert bl.sync_status() == "BL_ERR_NONFINITE"
    assert torch.equal(got[0], want[0]) and torch.equal(got[1, 2:], want[1, 2:])
    assert torch.isnan(got[1, :2]).all()


# ---- together ----------------------------------------------------------------------------------------------------------

def test_cached_steps_equal_the_prompt(bl):
    """A block's attention over ternary projections: the prompt through bl.attention, then token by token through
    the paged cache; the cached steps give what the whole prompt gives."""
    import torch
    n, hq, hk, d, kdim, page = 70, 4, 2, 64, 320, 16
    wide = (hq + 2 * hk) * d
    W, beta = bl.quantize_weights_pack5(normal(1, wide, kdim, scale=0.05))
    X = normal(2, n, kdim)
    table, gq, gk = bl.rope_table(n, d), 1 + 0.1 * normal(3, d), 1 + 0.1 * normal(4, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    Y = bl.linear(X, W, bl.PACK5, wide, kdim, beta)
    q, k, v = bl.qk_norm_rope(Y, hq, hk, d, pos, table, gq, gk)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, _ = bl.attention(q, k, v, cu, cu, n, window=40, sinks=2)
    kc, vc = (torch.full((8, hk, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = torch.tensor([[6, 1, 3, 0, 7]], dtype=torch.int32, device="cuda")
    ws = bl.workspace(bl.paged_attention_workspace_size(1, hq, kc), "cuda")
    for t in range(n):
        slot = pages[0, t // page].long() * page + t % page
        y = bl.linear(X[t:t + 1].contiguous(), W, bl.PACK5, wide, kdim, beta)
        qt = bl.qk_norm_rope_append(y, hq, hk, d, pos[t:t + 1], table, gq, gk, kc, vc, slot[None])
        assert torch.equal(qt[0], q[t])
        step = bl.paged_attention(qt, kc, vc, pages, torch.tensor([t + 1], dtype=torch.int32, device="cuda"), window=40,
                                  sinks=2, ws=ws)
        # the prompt's probabilities and result are rounded to bfloat16, the step's are not
        assert (step[0] - out[t].float()).abs().max() <= 2 * HALF["bfloat16"] * v[:t + 1].float().abs().max()
    ok(bl)


def test_training_step_gradients_by_differences(bl):
    """Projection -> norms, rotation -> attention -> a weighted sum: the chain of the library's gradients against
    differences of the float64 chain, along random directions of the projection's output and the gains."""
    import torch
    n, hq, hk, d = 60, 4, 2, 32
    Y, gq, gk = normal(1, n, (hq + 2 * hk) * d), 1 + 0.1 * normal(2, d), 1 + 0.1 * normal(3, d)
    w = normal(4, n, hq, d, dtype="float16")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table = bl.rope_table(n, d)
    cu = torch.tensor([0, 25, n], dtype=torch.int32, device="cuda")
    q, k, v = bl.qk_norm_rope(Y, hq, hk, d, pos, table, gq, gk, dtype=torch.float16)
    out, lse = bl.attention(q, k, v, cu, cu, 35, window=9, sinks=1)
    dq, dk, dv = bl.attention_backward(w, q, k, v, out, lse, cu, cu, 35, 35, window=9, sinks=1)
    dY, dgq, dgk = bl.qk_norm_rope_backward(dq, dk, dv, Y, hq, hk, d, pos, table, gq, gk)
    ok(bl)
    t, p, w8 = table.cpu().numpy(), pos.cpu().numpy(), f8(w)

    def loss(y, a, b):
        qq, kk, vv = split(y, hq, hk, d)
        qq, kk = A.norm_rope(qq, p, t, a, 1e-6), A.norm_rope(kk, p, t, b, 1e-6)
        return sum(float((A.attention(qq[s], kk[s], vv[s], 9, 1)[0] * w8[s]).sum()) for s in (slice(0, 25), slice(25, n)))
    x = [f8(Y), f8(gq), f8(gk)]
    rng = np.random.default_rng(0)
    for at, grad in enumerate((f8(dY), f8(dgq), f8(dgk))):
        for _ in range(3):
            step = rng.standard_normal(x[at].shape)
            up, down = list(x), list(x)
            up[at], down[at] = x[at] + 1e-5 * step, x[at] - 1e-5 * step
            got, want = float((grad * step).sum()), (loss(*up) - loss(*down)) / 2e-5
            # float16 on the way: each of the gradient's terms off by a few 2^-11, their signs independent
            assert abs(got - want) <= 40 * 2.0 ** -11 * np.linalg.norm(grad * step)


def test_other_stream_and_graph(bl):
    """The same results on another stream and from a captured graph replayed on new inputs."""
    import torch
    lens = [300, 77, 1000]
    q, kc, vc, pages, n, k, v = paged(4, lens, 8, 2, 64, 16, "bfloat16")
    ws = bl.workspace(bl.paged_attention_workspace_size(3, 8, kc), "cuda")
    fq, fk, fv, cq, ck = packed(7, [200, 133], [200, 133], 4, 2, 64, "float16")
    dout = normal(9, *fq.shape, dtype="float16")
    bws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    Y, pos, gq, gk = rows(5, 50, 4, 2, 64, 64)
    table = bl.rope_table(5000, 64)

    def run():
        a = bl.paged_attention(q, kc, vc, pages, n, ws=ws)
        out, lse = bl.attention(fq, fk, fv, cq, ck, 200, window=64, sinks=3)
        g = bl.attention_backward(dout, fq, fk, fv, out, lse, cq, ck, 200, 200, window=64, sinks=3, ws=bws)
        r = bl.qk_norm_rope(Y, 4, 2, 64, pos, table, gq, gk)
        b = bl.qk_norm_rope_backward(*r, Y, 4, 2, 64, pos, table, gq, gk, ws=bws)
        return [a, out, lse, *g, *r, *b]
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    q.copy_(q.flip(0))
    fq.copy_(fq.flip(0))
    Y.copy_(Y.flip(0))
    n.copy_(n.flip(0).clamp(max=int(n.min())))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(held, run()):
        assert torch.equal(x, y)
    ok(bl)


def test_two_streams_at_once(bl):
    """Calls that overlap on the GPU, each with a workspace of its own."""
    import torch
    lens = [3000, 77, 5000]
    a = paged(4, lens, 8, 2, 64, 16, "bfloat16")[:5]
    b = paged(9, lens, 8, 2, 64, 16, "bfloat16")[:5]
    f = packed(7, [900, 133], [900, 133], 4, 2, 64, "float16")
    dout = normal(9, *f[0].shape, dtype="float16")
    size = bl.paged_attention_workspace_size(3, 8, a[1])

    def step(x, ws):
        out, lse = bl.attention(*f, 900)
        return [bl.paged_attention(*x, ws=ws), out, *bl.attention_backward(dout, *f[:3], out, lse, *f[3:], 900, 900)]
    want = [step(x, bl.workspace(size, "cuda")) for x in (a, b)]
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [bl.workspace(size, "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = step(x, spaces[i])
    torch.cuda.synchronize()
    ok(bl)
    for x, y in zip(got, want):
        for s, t in zip(x, y):
            assert torch.equal(s, t)


def test_binding_refusals(bl):
    import torch
    q, k, v, cq, ck = packed(7, [20], [20], 4, 2, 64, "float16")
    with pytest.raises(ValueError):
        bl.attention(q.cpu(), k, v, cq, ck, 20)
    with pytest.raises(ValueError):
        bl.attention(q, k.bfloat16(), v, cq, ck, 20)
    with pytest.raises(ValueError):
        bl.attention(q.float(), k.float(), v.float(), cq, ck, 20)
    with pytest.raises(ValueError):
        bl.attention(q, k, v[:-1], cq, ck, 20)
    with pytest.raises(ValueError):
        bl.attention(q, k, v, cq.long(), ck, 20)
    with pytest.raises(ValueError):
        bl.attention(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cq, ck, 20)
    with pytest.raises(bl.BitLinearError):
        bl.attention(q, k.expand(20, 2, 64)[:1].expand(20, 2, 64), v, cq, ck, 20)    # rows on one another
    with pytest.raises(bl.BitLinearError):
        bl.attention(q, k, v, cq, ck, 20, window=-1)
    with pytest.raises(ValueError):
        bl.paged_attention(q, k, v, cq, ck)
    ok(bl)
