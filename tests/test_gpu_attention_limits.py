"""The attention operators on the GPU at the ends of their ranges, against the float64 oracle or a plain call."""
import numpy as np
import pytest

from oracle import attention as A
from test_gpu_attention import E, HALF, check_backward, check_forward, f8, normal, ok, packed, score_slack

pytestmark = pytest.mark.gpu
I32 = (1 << 31) - 1


@pytest.mark.parametrize("hq,hk", [(4, 2), (3, 1)])                  # two heads a CTA, two row blocks a CTA
def test_longest_lengths_may_be_any_upper_bound(bl, hq, hk):
    import torch
    q, k, v, cq, ck = packed(1, [150, 60], [150, 200], hq, hk, 64, "bfloat16")
    dout = normal(2, *q.shape, dtype="bfloat16")
    out, lse = bl.attention(q, k, v, cq, ck, 150)
    want = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, 150, 200)
    for most in (300, 1 << 30, I32 - 127, I32):
        got = bl.attention(q, k, v, cq, ck, most)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        grads = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, most, most)
        ok(bl)
        for n, (a, b) in enumerate(zip(grads, want)):
            # another bound may share out a group's heads otherwise, whose parts are then added in another order
            assert (a.float() - b.float()).abs().max() <= 2 * HALF["bfloat16"] * b.float().abs().max(), n
    check_forward(q, k, v, cq, ck, 0, 0, out, lse, "bfloat16")
    check_backward(q, k, v, cq, ck, 0, 0, out, lse, dout, grads, "bfloat16")


def test_paged_longest_length(bl):
    """Lengths up to 2^31 - 64 over a table that names one page again and again; longer ones are out of range."""
    import torch
    page, d, window, sinks = 1 << 17, 8, 100, 3
    kc, vc = (normal(n, 1, 1, page, d, dtype="bfloat16") for n in (1, 2))
    q = normal(3, 2, 1, d, dtype="bfloat16")
    table = torch.zeros(2, 1 << 14, dtype=torch.int32, device="cuda")
    most = (1 << 31) - 64
    lens = torch.tensor([most, 70], dtype=torch.int32, device="cuda")
    got = bl.paged_attention(q, kc, vc, table, lens, window=window, sinks=sinks)
    ok(bl)
    keys = [j % page for j in [*range(sinks), *range(most - window, most)]]
    for b, at in enumerate((keys, list(range(70)))):
        ro, _, p = A.attention(f8(q[b:b + 1]), f8(kc[0, 0, at])[:, None], f8(vc[0, 0, at])[:, None])
        # every key of the list is seen: the last one's query
        size = np.einsum("hj,jd->hd", p[:, 0], np.abs(f8(vc[0, 0, at])))
        tol = E * np.abs(ro[0]) + (score_slack(f8(q[b:b + 1]), f8(kc[0, 0, at])[:, None], d) + (len(at) + 40) * E) * size
        assert (np.abs(f8(got[b]) - ro[0]) <= tol).all()
    for n in (most + 1, I32):
        lens[0] = n
        again = bl.paged_attention(q, kc, vc, table, lens, window=window, sinks=sinks)
        assert bl.sync_status() == "BL_ERR_RANGE"
        assert torch.equal(again, got)


def gradients(bl, dout, q, k, v, scale=None):
    import torch
    n = q.shape[0]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = bl.attention(q, k, v, cu, cu, n, scale=scale)
    ok(bl)
    return bl.attention_backward(dout, q, k, v, out, lse, cu, cu, n, n, scale=scale)


@pytest.mark.parametrize("heads", [1, 2])                            # stored by the kernel itself; summed over two parts
def test_gradients_that_float16_does_not_reach_are_reported(bl, heads):
    import torch
    q, k, v = (normal(n, 1, h, 64, dtype="float16") for n, h in ((1, heads), (2, 1), (3, 1)))
    dout = torch.full_like(q, 65504.0 / heads)                        # one key: dV is the sum of dout over the heads
    dv = gradients(bl, dout, q, k, v)[2]
    ok(bl)
    assert (dv == 65504).all()
    dout[..., 5] = 32768.0 if heads == 2 else 65504.0
    dv = gradients(bl, dout, q, k, v)[2]
    # 65504 is reached, 65536 is not
    assert bl.sync_status() == ("BL_ERR_NONFINITE" if heads == 2 else "BL_OK")
    assert torch.isinf(dv[..., 5]).all() == (heads == 2) and (dv[..., :5] == 65504).all()


def test_sums_over_queries_that_float16_does_not_reach_are_reported(bl):
    import torch
    n = 300
    q, k, v = (torch.zeros(n, 1, 64, dtype=torch.float16, device="cuda") for _ in range(3))
    q[..., 0], k[0, 0, 0] = 8.0, 16.0                                 # every query sees the first key with weight 1 - 2^-14
    dv = gradients(bl, torch.full_like(q, 300.0), q, k, v)[2]
    assert bl.sync_status() == "BL_ERR_NONFINITE"
    assert torch.isinf(dv[0]).all() and torch.isfinite(dv[1:]).all()
    # the second query's keys are +-60, its probabilities 1/2 each, dP = +-6400: dQ = 2 * 3200 * 60
    q, k, v = (torch.zeros(2, 1, 64, dtype=torch.float16, device="cuda") for _ in range(3))
    k[0], k[1], v[0], v[1] = 60.0, -60.0, 1.0, -1.0
    dq, dk, dv = gradients(bl, torch.full_like(q, 100.0), q, k, v, scale=1.0)
    assert bl.sync_status() == "BL_ERR_NONFINITE"
    assert torch.isinf(dq[1]).all() and torch.isfinite(dk).all() and torch.isfinite(dv).all()
    dq, _, _ = gradients(bl, torch.full_like(q, 100.0), q, k, v, scale=0.125)
    ok(bl)
    assert (dq[1] == 48000).all() and not dq[0].any()


NORMS = [(3, 2, 1, 32), (5000, 16, 8, 32)]                           # a kernel of single heads; one fed by bulk copies


@pytest.mark.parametrize("m,hq,hk,d", NORMS)
@pytest.mark.parametrize("dtype,past", [("float16", 65520.0), ("bfloat16", 3.4e38)])
def test_values_that_the_type_does_not_reach_are_reported(bl, m, hq, hk, d, dtype, past):
    import torch
    from test_gpu_attention import rows
    qkv, pos, gq, gk = rows(8, m, hq, hk, d, d)
    table, t, v0 = bl.rope_table(5000, d), getattr(torch, dtype), (hq + hk) * d
    biggest = torch.finfo(t).max

    def both():
        cache = [torch.zeros(m, hk, 1, d, dtype=t, device="cuda") for _ in range(2)]
        yield lambda: bl.qk_norm_rope(qkv, hq, hk, d, pos, table, gq, gk, dtype=t)[2]
        yield lambda: (bl.qk_norm_rope_append(qkv, hq, hk, d, pos, table, gq, gk, *cache, torch.arange(m, device="cuda")),
                       cache[1][:, :, 0])[1]
    for f in both():
        qkv[m - 1, v0:v0 + 8] = biggest
        f()
        ok(bl)
        qkv[m - 1, v0 + 5] = past
        v = f()
        assert bl.sync_status() == "BL_ERR_NONFINITE"
        assert torch.isinf(v[m - 1, 0, 5]) and torch.isfinite(v[:m - 1]).all()


@pytest.mark.parametrize("m,hq,hk,d", NORMS)
@pytest.mark.parametrize("dtype,gain", [("float16", 1e5), ("bfloat16", 3.39e38), ("float32", 3.39e38)])
def test_normed_heads_that_the_type_does_not_reach_are_reported(bl, m, hq, hk, d, dtype, gain):
    import torch
    from test_gpu_attention import rows
    qkv, pos, gq, gk = rows(8, m, hq, hk, d, d)
    qkv[m - 1, hq * d:(hq + hk) * d] = 0.0
    qkv[m - 1, hq * d + 3] = 1.0                                      # normed: the root of d
    gk[3] = gain
    gk[:3], gk[4:] = 0.0, 0.0
    qkv[:m - 1, hq * d:(hq + hk) * d].view(m - 1, hk, d)[..., 3] = 0.0
    k = bl.qk_norm_rope(qkv, hq, hk, d, pos, None, gq, gk, dtype=getattr(torch, dtype))[1]
    assert bl.sync_status() == "BL_ERR_NONFINITE"
    assert torch.isinf(k[m - 1, 0, 3]) and not k[:m - 1].any()


@pytest.mark.parametrize("sign", [1, -1])
def test_averages_of_the_largest_values_stay_finite(bl, sign):
    """P is rounded for the tensor cores, its sum is not: the average of equal values may come out up to 2^-11 larger."""
    import torch
    n, d = 257, 64
    q, k = (torch.zeros(n, 1, d, dtype=torch.float16, device="cuda") for _ in range(2))
    q[:, 0, 0] = torch.linspace(0.01, 3, n)
    k[0, 0, 0] = 8.0                                                  # one key far above the others, which all round alike
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for value in (65504.0, 65472.0, 1.0):
        v = torch.full_like(k, sign * value)
        out, _ = bl.attention(q, k, v, cu, cu, n)
        ok(bl)
        assert (out.float() - sign * value).abs().max() <= value * 1.5 * 2.0 ** -10    # P's rounding and the result's
    v[5, 0, 7] = float("inf")
    out, _ = bl.attention(q, k, v, cu, cu, n)
    assert bl.sync_status() == "BL_ERR_NONFINITE" and torch.isinf(out[6:, 0, 7]).all()
    big = torch.full_like(k, 3e38, dtype=torch.bfloat16)              # their sum passes float32 in no row of one key
    out, _ = bl.attention(q[:1].bfloat16(), k[:1].bfloat16(), big[:1], cu.clamp(max=1), cu.clamp(max=1), 1)
    ok(bl)
    assert torch.equal(out, big[:1])


@pytest.mark.parametrize("m,hq,hk,d", NORMS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_norm_gradients_report_what_is_not_finite(bl, m, hq, hk, d, dtype):
    """A NaN or Inf in any of the gradients that come in, and a gradient that passes float32 on the way."""
    import torch
    from test_gpu_attention import rows
    qkv, pos, gq, gk = rows(8, m, hq, hk, d, d)
    table = bl.rope_table(5000, d)
    grads = [normal(n, m, h, d, dtype=dtype) for n, h in ((3, hq), (4, hk), (5, hk))]
    want = bl.qk_norm_rope_backward(*grads, qkv, hq, hk, d, pos, table, gq, gk)
    ok(bl)
    for n in range(3):
        for bad in (float("nan"), float("-inf")):
            use = [g.clone() for g in grads]
            use[n][m - 1, -1, d - 1] = bad
            dx, _, _ = bl.qk_norm_rope_backward(*use, qkv, hq, hk, d, pos, table, gq, gk)
            assert bl.sync_status() == "BL_ERR_NONFINITE", (n, bad)
            assert torch.equal(dx[:m - 1], want[0][:m - 1])
    use = [g.clone() for g in grads]
    use[0][m - 1] = 3e38                                              # finite; its products with the gains and 1/rms are not
    small = qkv.clone()
    small[m - 1] *= 1e-6
    bl.qk_norm_rope_backward(*use, small, hq, hk, d, pos, table, gq, gk)
    assert bl.sync_status() == "BL_ERR_NONFINITE"


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_scores_far_below_zero(bl, window, sinks):
    """Scores down to -2^113 are scores like others: a row's largest takes it all."""
    import torch
    n, d = 300, 64
    q, k = (torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[..., 0] = 2.0 ** 58
    at = (np.arange(n) * 37) % 251 + 1                                # whole numbers below 2^8, alike 251 apart only
    k[:, 0, 0] = torch.from_numpy(-(2.0 ** 50) * at).cuda()
    v = normal(1, n, 1, d, dtype="bfloat16")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = bl.attention(q, k, v, cu, cu, n, window=window, sinks=sinks)
    ok(bl)
    see = A.visible(n, n, window, sinks)
    weight = np.where(see, at, 1000)
    weight = weight == weight.min(1, keepdims=True)
    want = (weight / weight.sum(1, keepdims=True)) @ f8(v[:, 0])
    assert (np.abs(f8(out[:, 0]) - want) <= 1.01 * HALF["bfloat16"] * np.abs(want)).all()
    assert (np.abs(f8(lse[0]) / (-(2.0 ** 105) * np.where(see, at, 1000).min(1)) - 1) <= 4 * E).all()
    pages = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")
    cache = [torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 4)).reshape(-1, 16, 1, d).transpose(1, 2).contiguous() for t in (k, v)]
    lens = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
    got = bl.paged_attention(q, *cache, pages.expand(n, -1).contiguous(), lens, window=window, sinks=sinks)
    ok(bl)
    assert (np.abs(f8(got[:, 0]) - want) <= 8 * E * np.abs(want)).all()


def test_scores_that_pass_float32_are_reported(bl):
    import torch
    n, d = 3, 64
    q, k = (torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[1, 0, 0], k[:, 0, 0] = 1e20, -1e20                              # the second row's scores are all -1e40
    v, cu = normal(1, n, 1, d, dtype="bfloat16"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, _ = bl.attention(q, k, v, cu, cu, n)
    assert bl.sync_status() == "BL_ERR_NONFINITE"
    assert torch.equal(out[0], v[0])
    cache = [torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 13)).reshape(1, 16, 1, d).transpose(1, 2).contiguous() for t in (k, v)]
    bl.paged_attention(q[1:2].contiguous(), *cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                       torch.tensor([2], dtype=torch.int32, device="cuda"))
    assert bl.sync_status() == "BL_ERR_NONFINITE"


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gradients_do_not_depend_on_what_a_sequence_is_packed_with(bl, dtype):
    """Sequences and heads whose gradients are 2^20 apart: each comes out as if it were alone, bit for bit."""
    import torch
    lens, h, d = [512, 300, 129], 3, 64                               # a head a key head: nothing is shared out
    q, k, v, cu, _ = packed(5, lens, lens, h, h, d, dtype)
    size = torch.ones(sum(lens), h, 1, device="cuda")
    size[512:812], size[812:, 1] = 2.0 ** 10, 2.0 ** 10
    size[:512] = 2.0 ** -10
    dout = (normal(6, *q.shape) * size).to(q.dtype)
    out, lse = bl.attention(q, k, v, cu, cu, 512, window=200, sinks=2)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cu, cu, 512, 512, window=200, sinks=2)
    ok(bl)
    check_backward(q, k, v, cu, cu, 200, 2, out, lse, dout, grads, dtype)
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for head in range(h):
            f = lambda t: t[rows, head:head + 1].contiguous()  # noqa: E731,B023
            alone = bl.attention_backward(f(dout), f(q), f(k), f(v), f(out), lse[head:head + 1, rows].contiguous(), one, one, n, n,
                                          window=200, sinks=2)
            for x, y in zip(grads, alone):
                assert torch.equal(f(x), y)
    ok(bl)


def test_gradients_of_many_short_sequences(bl):
    import torch
    rng = np.random.default_rng(1)
    lq = rng.integers(0, 4, 700).tolist()
    lk = [n + int(rng.integers(0, 3)) for n in lq]
    q, k, v, cq, ck = packed(5, lq, lk, 6, 3, 32, "float16")
    dout = (normal(6, *q.shape) * torch.logspace(-2, 2, q.shape[0], device="cuda")[:, None, None]).half()
    out, lse = bl.attention(q, k, v, cq, ck, 3)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, 3, 5)
    ok(bl)
    check_forward(q, k, v, cq, ck, 0, 0, out, lse, "float16")
    check_backward(q, k, v, cq, ck, 0, 0, out, lse, dout, grads, "float16")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gradients_of_many_heads_a_key_head(bl, dtype):
    """More heads than rows that a CTA of the row sums takes; more keys than queries, and fewer."""
    q, k, v, cq, ck = packed(5, [9, 70, 200], [300, 70, 40], 96, 1, 64, dtype)
    dout = normal(6, *q.shape, dtype=dtype)
    out, lse = bl.attention(q, k, v, cq, ck, 200)
    grads = bl.attention_backward(dout, q, k, v, out, lse, cq, ck, 200, 300)
    ok(bl)
    check_backward(q, k, v, cq, ck, 0, 0, out, lse, dout, grads, dtype)


def dirty(*shapes):
    """Fills the allocator's free blocks of these sizes with NaN."""
    import torch
    held = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in shapes for _ in range(8)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("dtype,hq,hk", [("bfloat16", 4, 2), ("float16", 3, 3)])
def test_rows_of_no_sequence_are_clear_in_new_outputs(bl, dtype, hq, hk):
    """Padding before and behind the sequences: outputs of the allocator hold zeros there (lse -inf), and a gain's
    gradient, summed over all rows, is that of the sequences alone."""
    import torch
    d, lo, n, more = 64, 40, 300, 5000
    T = lo + n + more
    Y = normal(1, T, (hq + 2 * hk) * d)
    table, gq, gk = bl.rope_table(T, d), 1 + 0.1 * normal(2, d), 1 + 0.1 * normal(3, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    q, k, v = bl.qk_norm_rope(Y, hq, hk, d, pos, table, gq, gk, dtype=getattr(torch, dtype))
    cu = torch.tensor([lo, lo + 120, lo + n], dtype=torch.int32, device="cuda")
    one = cu - lo
    w = normal(4, *q.shape, dtype=dtype)
    shapes = [((T, h, d), q.dtype) for h in (hq, hk)] + [((hq, T), torch.float32)]
    dirty(*shapes)
    out, lse = bl.attention(q, k, v, cu, cu, 180)
    ok(bl)
    own = slice(lo, lo + n)
    f = lambda t: t[own].contiguous()  # noqa: E731
    o1, l1 = bl.attention(f(q), f(k), f(v), one, one, 180)
    assert torch.equal(out[own], o1) and torch.equal(lse[:, own], l1)
    for rest in (slice(0, lo), slice(lo + n, T)):
        assert not out[rest].any() and (lse[:, rest] == -float("inf")).all()
    dirty(*shapes)
    grads = bl.attention_backward(w, q, k, v, out, lse, cu, cu, 180, 180)
    alone = bl.attention_backward(f(w), f(q), f(k), f(v), o1, l1, one, one, 180, 180)
    ok(bl)
    for a, b in zip(grads, alone):
        assert torch.equal(a[own], b) and not a[:lo].any() and not a[lo + n:].any()
    dY, dgq, dgk = bl.qk_norm_rope_backward(*grads, Y, hq, hk, d, pos, table, gq, gk)
    eY, egq, egk = bl.qk_norm_rope_backward(*alone, f(Y), hq, hk, d, f(pos), table, gq, gk)
    ok(bl)
    assert torch.equal(dY[own], eY) and not dY[:lo].any() and not dY[lo + n:].any()
    for x, y in ((dgq, egq), (dgk, egk)):                             # other partial sums, of at most n * heads terms
        assert (x - y).abs().max() <= 2 * n * hq * E * y.abs().max() * 8


def test_no_sequence_at_all_gives_clear_outputs(bl):
    import torch
    q, k = normal(1, 50, 4, 64, dtype="bfloat16"), normal(2, 70, 2, 64, dtype="bfloat16")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    shapes = [((50, 4, 64), q.dtype), ((70, 2, 64), q.dtype), ((4, 50), torch.float32)]
    for c in (cu, torch.zeros(3, dtype=torch.int32, device="cuda")):    # none; two empty ones
        dirty(*shapes)
        out, lse = bl.attention(q, k, k, c, c, 0)
        assert not out.any() and (lse == -float("inf")).all()
        dirty(*shapes)
        grads = bl.attention_backward(q, q, k, k, out, lse, c, c, 0, 0)
        ok(bl)
        assert not any(g.any() for g in grads)
    held = torch.full_like(q, 3.0)
    assert (bl.attention(q, k, k, cu, cu, 0, out=held)[0] == 3).all()
    ok(bl)


def test_the_status_word_read_is_that_of_the_calls(bl, tmp_path):
    """In a process of its own, with a copy of the library: an error of an attention call is seen."""
    import os
    import shutil
    import subprocess
    import sys
    copy = shutil.copy(bl.LIB_PATH, tmp_path / "libother.so")
    code = ("import torch, int8_row_absmax_b200 as bl\n"
            f"bl.load({str(copy)!r})\n"
            "q = torch.zeros(4, 1, 64, dtype=torch.float16, device='cuda')\n"
            "cu = torch.tensor([0, 4], dtype=torch.int32, device='cuda')\n"
            "bl.attention(q, q, q, cu, cu, 4)\n"
            "assert bl.sync_status() == 'BL_OK'\n"
            "bl.attention(q, q, q, cu, cu, 2)\n"
            "assert bl.sync_status() == 'BL_ERR_RANGE'\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(bl.PKG_DIR), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("dtype,hq,hk,d,window,sinks", [("bfloat16", 2, 2, 96, 128, 65), ("float16", 12, 3, 96, 200, 4),
                                                        ("bfloat16", 8, 2, 64, 0, 0), ("float16", 3, 1, 128, 0, 0)])
def test_results_do_not_depend_on_what_a_sequence_is_packed_with(bl, dtype, hq, hk, d, window, sinks):
    """The rows behind a sequence's end lie in its last tile: large ones, or infinities, change no bit of its results."""
    import torch
    lq, lk = [266, 26, 150, 140], [266, 529, 290, 900]
    q, k, v, cq, ck = packed(3, lq, lk, hq, hk, d, dtype, scale=3.0)
    q[292:442] *= 8                                                   # the third sequence's scores: far larger
    alone = []
    for b in range(4):
        f = lambda t, c: t[int(c[b]):int(c[b + 1])].contiguous()  # noqa: E731,B023
        one = [torch.tensor([0, n[b]], dtype=torch.int32, device="cuda") for n in (lq, lk)]
        alone.append(bl.attention(f(q, cq), f(k, ck), f(v, ck), *one, lq[b], window=window, sinks=sinks))
    wide = [torch.cat([t, torch.full((200, *t.shape[1:]), float("inf"), dtype=t.dtype, device="cuda")]) for t in (q, k, v)]
    for x in ((q, k, v), wide):
        out, lse = bl.attention(*x, cq, ck, 266, window=window, sinks=sinks)
        ok(bl)
        for b in range(4):
            rows = slice(int(cq[b]), int(cq[b + 1]))
            assert torch.equal(out[rows], alone[b][0]) and torch.equal(lse[:, rows], alone[b][1])


@pytest.mark.parametrize("dtype,size", [("float16", 2.0 ** 10), ("float16", 2.0 ** 15), ("bfloat16", 2.0 ** 12), ("bfloat16", 2.0 ** 20),
                                        ("bfloat16", 2.0 ** 40), ("bfloat16", 2.0 ** 100)])
@pytest.mark.parametrize("sign,window", [(1, 0), (-1, 0), (1, 100), (-1, 100)])
def test_scores_of_any_size(bl, dtype, size, sign, window):
    """Scores up to 2^29 (float16) and 2^114 apart: the exact product of a score and its scale, less the rounded row
    maximum, would pass what a probability has room for."""
    import torch
    n, d = 300, 64
    q, k = (torch.zeros(n, 1, d, dtype=getattr(torch, dtype), device="cuda") for _ in range(2))
    at = (np.arange(n) * 37) % 251 + 1
    q[..., 0], k[:, 0, 0] = size, torch.from_numpy(64.0 * sign * at).cuda()
    v = normal(1, n, 1, d, dtype=dtype)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = bl.attention(q, k, v, cu, cu, n, window=window, scale=1.0)
    ok(bl)
    score = np.where(A.visible(n, n, window), sign * at * 64.0 * size, -np.inf)
    best = score == score.max(1, keepdims=True)                       # the next one is 2^16 less at least
    want = (best / best.sum(1, keepdims=True)) @ f8(v[:, 0])
    assert (np.abs(f8(out[:, 0]) - want) <= 1.01 * HALF[dtype] * np.abs(want)).all()
    assert (np.abs(f8(lse[0]) / (score.max(1) + np.log(best.sum(1))) - 1) <= 4 * E).all()


def test_a_captured_step_takes_other_bounds(bl):
    """One graph for every batch that fits the buffers: bounds are read on the device, and the rows that they leave are
    cleared on each replay."""
    import torch
    T, hq, hk, d = 700, 4, 2, 64
    q, k, v = (normal(n, T, h, d, dtype="float16") for n, h in ((1, hq), (2, hk), (3, hk)))
    dout = normal(4, T, hq, d, dtype="float16")
    cu = torch.tensor([0, 400, 500, 700], dtype=torch.int32, device="cuda")

    def step():
        out, lse = bl.attention(q, k, v, cu, cu, T, window=150, sinks=2)
        return out, lse, *bl.attention_backward(dout, q, k, v, out, lse, cu, cu, T, T, window=150, sinks=2)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for bounds in ([0, 400, 500, 700], [10, 10, 300, 333], [5, 260, 261, 262], [0, 0, 0, 0], [0, 1, 699, 700]):
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        for t in held:
            t.fill_(7.0)
        graph.replay()
        want = step()
        ok(bl)
        for a, b in zip(held, want):
            assert torch.equal(a, b)
        lo, hi = bounds[0], bounds[-1]
        for rest in (slice(0, lo), slice(hi, T)):
            assert not any(held[i][rest].any() for i in (0, 2, 3, 4)) and (held[1][:, rest] == -float("inf")).all()
        check_forward(q, k, v, cu, cu, 150, 2, held[0], held[1], "float16")
