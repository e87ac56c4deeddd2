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
