"""Host-side limits of the attention operators: sizes at the ends of their types."""
import ctypes

import pytest

import int8_row_absmax_b200 as pkg
from int8_row_absmax_b200 import attn
from int8_row_absmax_b200 import build as blbuild

I32 = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    blbuild.build()
    return pkg.load()


def call(**kw):
    d = dict(t=2, Hq=4, Hkv=2, D=64, q=16, k=16, v=16, ldq=256, ldk=128, ldv=128, Tq=10, Tk=10, cu_q=16, cu_k=16, B=1,
             max_q=10, max_k=10, window=0, sinks=0, scale=0.125)
    d.update(kw)
    return ctypes.byref(attn.AttnCall(**d))


@pytest.mark.parametrize("most", [11, 1000, 1 << 30, I32 - 127, I32])
def test_a_longest_length_past_the_buffer_counts_as_the_buffer(lib, most):
    """Blocks of rows are counted from the longest length in 32 bits: it is bounded by the buffer's rows first."""
    size = lib.bl_attention_backward_workspace_size
    assert size(call(max_q=most, max_k=most)) == size(call())
