"""The attention operators on the GPU where there is much of something: the norms' kernels that are fed by bulk copies
(each test asks the library which kernel its rows take), tens of blocks a sequence, offsets past 32 bits, and every
counter of the paged kernel's workspace."""
import ctypes

import numpy as np
import pytest

from test_gpu_attention import check_backward, check_forward, f8, normal, ok, packed, paged, rows

pytestmark = pytest.mark.gpu


def by_copies(bl, qkv, hq, hk, d, backward=0):
    """Whether rows [M, (hq + 2 hk) d] go through a kernel that is fed by bulk copies."""
    p = qkv.data_ptr()
    r = bl.QkvRows(M=qkv.shape[0], Hq=hq, Hkv=hk, D=d, q=p, k=p, v=p, ldq=qkv.shape[1], ldk=qkv.shape[1], ldv=qkv.shape[1],
                   eps=1e-6)
    return bl.load().bl_qk_norm_rope_plan(ctypes.byref(r), backward, None) == 1


SHAPES = [(4801, 12, 2, 64, 64, False, "float16"), (4900, 12, 3, 32, 16, True, "bfloat16"), (1600, 20, 5, 128, 128, False, "bfloat16"),
          (1300, 12, 3, 256, 64, True, "float16"), (4800, 6, 1, 80, 80, False, "bfloat16")]


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dtype", SHAPES)
def test_append_by_copies(bl, m, hq, hk, d, rot, inter, dtype):
    """Equal, bit for bit, to the kernel of single heads on the same rows; slots out of order, some rows without one."""
    import torch
    qkv, pos, gq, gk = rows(m, m, hq, hk, d, rot)
    table, t, page = bl.rope_table(5000, rot), getattr(torch, dtype), 24
    n = -(-m // page) + 3
    kc, vc = (normal(i, n, hk, page, d, dtype=dtype) for i in (1, 2))
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.from_numpy(np.random.default_rng(1).permutation(n * page)[:m]).cuda()
    slots[7::100] = -1
    assert by_copies(bl, qkv, hq, hk, d) and not by_copies(bl, qkv[:100], hq, hk, d)
    q = bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, kc, vc, slots, interleaved=inter)
    q0 = torch.cat([bl.qk_norm_rope_append(qkv[i:i + 100], hq, hk, d, pos[i:i + 100], table, gq, gk, k0, v0, slots[i:i + 100],
                                           interleaved=inter) for i in range(0, m, 100)])
    ok(bl)
    assert torch.equal(q, q0) and torch.equal(kc, k0) and torch.equal(vc, v0)
    k1, v1 = (bl.qk_norm_rope(qkv, hq, hk, d, pos, table, gq, gk, dtype=t, interleaved=inter)[i] for i in (1, 2))
    keep = slots >= 0
    assert torch.equal(kc[slots[keep] // page, :, slots[keep] % page], k1[keep])
    assert torch.equal(vc[slots[keep] // page, :, slots[keep] % page], v1[keep])


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dtype", SHAPES)
def test_bad_positions_and_slots_by_copies(bl, m, hq, hk, d, rot, inter, dtype):
    """Reported; what they would have addressed is not written, all else is."""
    import torch
    qkv, pos, gq, gk = rows(m, m, hq, hk, d, rot)
    table, t, page = bl.rope_table(5000, rot), getattr(torch, dtype), 16
    n = -(-m // page)
    assert by_copies(bl, qkv, hq, hk, d)
    slots = torch.arange(m, device="cuda")
    bad = {0: (-1, 0), 5: (5000, 5), m // 2: (1, n * page), m // 2 + 1: (1, 1 << 40), m - 1: (2 ** 31 - 1, m - 1)}

    def run():
        kc, vc = (torch.full((n, hk, page, d), 3.0, dtype=t, device="cuda") for _ in range(2))
        q = bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, kc, vc, slots, interleaved=inter)
        return q, *(c.transpose(1, 2).reshape(n * page, hk, d)[:m] for c in (kc, vc))
    want = run()
    ok(bl)
    for i, (p, s) in bad.items():
        pos[i], slots[i] = p, s
    got = run()
    assert bl.sync_status() == "BL_ERR_RANGE"
    good = torch.ones(m, dtype=torch.bool, device="cuda")
    good[list(bad)] = False
    assert torch.equal(got[0][good], want[0][good])
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[good], b[good]) and (a[~good] == 3).all()


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dtype", SHAPES)
def test_what_is_not_finite_by_copies(bl, m, hq, hk, d, rot, inter, dtype):
    import torch
    qkv, pos, gq, gk = rows(m, m, hq, hk, d, rot)
    table, t = bl.rope_table(5000, rot), getattr(torch, dtype)
    assert by_copies(bl, qkv, hq, hk, d)
    f = lambda x: bl.qk_norm_rope(x, hq, hk, d, pos, table, gq, gk, dtype=t, interleaved=inter)  # noqa: E731
    want = f(qkv)
    ok(bl)
    for row, col, value in ((0, 3, "nan"), (m - 1, hq * d + 1, "inf"), (m // 2, (hq + hk) * d + 5, "-inf"), (9, (hq + 2 * hk) * d - 1, "nan")):
        x = qkv.clone()
        x[row, col] = float(value)
        got = f(x)
        assert bl.sync_status() == "BL_ERR_NONFINITE", (row, col)
        keep = torch.arange(m, device="cuda") != row
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep])
    if dtype == "bfloat16":                                           # a value's square may overflow: values are only converted
        x = qkv.clone()
        x[m - 1, (hq + hk) * d:] = 1e25
        v = f(x)[2]
        ok(bl)
        assert torch.equal(v[m - 1].flatten(), x[m - 1, (hq + hk) * d:].bfloat16())


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dtype", SHAPES)
def test_norm_gradients_by_copies_repeat_and_leave_out_bad_positions(bl, m, hq, hk, d, rot, inter, dtype):
    import torch
    qkv, pos, gq, gk = rows(m, m, hq, hk, d, rot)
    table = bl.rope_table(5000, rot)
    grads = [normal(n, m, h, d, dtype=dtype) for n, h in ((3, hq), (4, hk), (5, hk))]
    assert by_copies(bl, qkv, hq, hk, d, 1)
    f = lambda g, p: bl.qk_norm_rope_backward(*g, qkv, hq, hk, d, p, table, gq, gk, interleaved=inter)  # noqa: E731
    one, two = f(grads, pos), f(grads, pos)
    ok(bl)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    at = [0, 17, m - 1]
    out = [g.clone() for g in grads]
    for g in out:
        g[at] = 0.0
    want = f(out, pos)
    ok(bl)
    bad = pos.clone()
    bad[at] = torch.tensor([-1, 5000, 1 << 30], dtype=torch.int32, device="cuda")
    got = f(grads, bad)
    assert bl.sync_status() == "BL_ERR_RANGE"
    good = torch.ones(m, dtype=torch.bool, device="cuda")
    good[at] = False
    assert torch.equal(got[0][good], one[0][good])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("lens,hq,hk,d", [([2000, 1500], 32, 8, 128), ([9000], 2, 1, 64), ([40000, 3, 40000], 40, 1, 32)])
def test_paged_workspace_is_left_clear(bl, lens, hq, hk, d):
    q, kc, vc, pages, n, _, _ = paged(1, lens, hq, hk, d, 64, "bfloat16")
    ws = bl.workspace(bl.paged_attention_workspace_size(len(lens), hq, kc), "cuda")
    for _ in range(3):
        bl.paged_attention(q, kc, vc, pages, n, ws=ws)
        ok(bl)
        assert not ws[:4 * 592].any()                                 # a counter for each of four CTAs on 148 SMs


@pytest.mark.parametrize("n,hq,hk,d,window,sinks,dtype", [(5003, 2, 1, 64, 0, 0, "float16"), (4500, 2, 1, 128, 0, 0, "bfloat16"),
                                                          (5003, 3, 1, 128, 1700, 130, "bfloat16"), (3333, 2, 2, 32, 2000, 1, "float16")])
def test_tens_of_blocks(bl, n, hq, hk, d, window, sinks, dtype):
    lens = [n, 70]
    q, k, v, cq, ck = packed(n, lens, [n + 111, 70], hq, hk, d, dtype)
    out, lse = bl.attention(q, k, v, cq, ck, n, window=window, sinks=sinks)
    dout = normal(99, *q.shape, dtype=dtype)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, n, n + 111, window=window, sinks=sinks)
    ok(bl)
    check_forward(q, k, v, cq, ck, window, sinks, out, lse, dtype)
    check_backward(q, k, v, cq, ck, window, sinks, out, lse, dout, grads, dtype)


@pytest.mark.parametrize("hq,hk", [(32, 32), (32, 4)])               # 4: a key block's heads are shared out
def test_packed_rows_past_32_bit_offsets(bl, hq, hk):
    """Sequences behind 2^31 elements of rows that belong to none: bit for bit what they are at the buffers' start."""
    import torch
    d, lens = 128, [200, 70]
    q, k, v, cu, _ = packed(1, lens, lens, hq, hk, d, "bfloat16")
    dout = normal(2, *q.shape, dtype="bfloat16")
    lo, n = (1 << 31) // (32 * d) + 10, sum(lens)

    def far(t):
        wide = torch.zeros(lo + n, *t.shape[1:], dtype=t.dtype, device="cuda")
        wide[lo:] = t
        return wide
    out, lse = bl.attention(q, k, v, cu, cu, 200)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cu, cu, 200, 200)
    Q, K, V, G = (far(t) for t in (q, k, v, dout))
    O, L = bl.attention(Q, K, V, cu + lo, cu + lo, 200)
    ok(bl)
    assert torch.equal(O[lo:], out) and torch.equal(L[:, lo:], lse)
    assert not O[:lo].any() and (L[:, :lo] == -float("inf")).all()
    got = bl.attention_backward(G, Q, K, V, O, L, cu + lo, cu + lo, 200, 200)
    ok(bl)
    for a, b in zip(got, grads):
        assert torch.equal(a[lo:], b) and not a[:lo].any()
    del Q, K, V, G, O, L, got
    torch.cuda.empty_cache()


def test_strided_rows_past_32_bit_offsets(bl):
    """Tokens 2^23 elements apart."""
    import torch
    n, hq, hk, d = 300, 4, 2, 64
    wide = torch.zeros(n, 1 << 23, dtype=torch.float16, device="cuda")
    q, k, v, cu, _ = packed(1, [n], [n], hq, hk, d, "float16")
    parts = [(q, 8), (k, 4096), (v, (1 << 23) - hk * d)]
    views = [wide[:, c:c + t.shape[1] * d].unflatten(1, t.shape[1:]) for t, c in parts]
    for t, view in zip((q, k, v), views):
        view.copy_(t)
    want, got = bl.attention(q, k, v, cu, cu, n), bl.attention(*views, cu, cu, n)
    dout = normal(2, *q.shape, dtype="float16")
    g0, g1 = (bl.attention_backward(dout, *x, *want, cu, cu, n, n) for x in ((q, k, v), views))
    ok(bl)
    for a, b in zip((*want, *g0), (*got, *g1)):
        assert torch.equal(a, b)
    check_forward(q, k, v, cu, cu, 0, 0, *got, "float16")
    assert np.isfinite(f8(g1[0])).all()
    del wide, views
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_loose_longest_lengths_of_many_sequences(bl, dtype):
    """Lengths known only as at most the buffer's, a thousand sequences: the calls take them, and soon."""
    import torch
    lens = np.random.default_rng(1).integers(1, 40, 1000).tolist()
    q, k, v, cu, _ = packed(1, lens, lens, 32, 8, 64, dtype)
    dout = normal(2, *q.shape, dtype=dtype)
    out, lse = bl.attention(q, k, v, cu, cu, 40)
    want = bl.attention_backward(dout, q, k, v, out, lse, cu, cu, 40, 40)
    loose = q.shape[0]
    got = bl.attention(q, k, v, cu, cu, loose)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    for a, b in zip(bl.attention_backward(dout, q, k, v, out, lse, cu, cu, loose, loose), want):
        assert torch.equal(a, b)
    ok(bl)
    one = slice(int(cu[500]), int(cu[501]))
    first = torch.tensor([0, lens[500]], dtype=torch.int32, device="cuda")
    check_forward(q[one], k[one], v[one], first, first, 0, 0, out[one], lse[:, one], dtype)
    check_backward(q[one], k[one], v[one], first, first, 0, 0, out[one], lse[:, one], dout[one], [g[one] for g in want], dtype)
