"""The attention operators on the GPU at the ends of their ranges, against the float64 oracle or a plain call."""
import numpy as np
import pytest

from oracle import attention as A
from test_gpu_attention import E, HALF, check_backward, check_forward, f8, normal, ok, packed

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
