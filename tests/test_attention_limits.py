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


def test_clearing_refusals(lib):
    """Which outputs may be cleared by which call, and that what is to be cleared is there."""
    f, b = lib.bl_attention_ex, lib.bl_attention_backward_ex
    none = dict(B=0, q=None, k=None, v=None, cu_q=None, cu_k=None)
    assert f(call(), 16, 16, 4, None) == 1 and f(call(), 16, 16, 64, None) == 1 and f(call(), 16, None, 2, None) == 1
    assert f(call(**none), None, 16, 1, None) == 1 and f(call(**none), 16, None, 3, None) == 1
    assert f(call(**none), 24, 16, 3, None) == 2
    assert f(call(**none), None, None, 0, None) == 0 and f(call(Tq=0, q=None), None, None, 3, None) == 0
    args = [16, 16, 16, 16, 16, 16, 256, 1 << 30]
    assert b(call(), *args, 1, None) == 1 and b(call(), *args, 32, None) == 1
    for at, bit in ((3, 4), (4, 8), (5, 16)):
        bad = list(args)
        bad[at] = None
        assert b(call(**none), *bad, bit, None) == 1
        bad[at] = 24
        assert b(call(**none), *bad, bit, None) == 2
    assert b(call(**none), *[None] * 7, 0, 0, None) == 0


def rows(**kw):
    d = dict(M=2, Hq=32, Hkv=8, D=128, q=256, k=256, v=256, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, pos=256, table=256, P=10, R=0,
             interleaved=0, gq=None, gk=None, eps=1e-6)
    d.update(kw)
    return ctypes.byref(attn.QkvRows(**d))


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("d", [8, 24, 32, 40, 56, 64, 80, 96, 128, 160, 256])
def test_many_rows_take_no_more_ctas_than_run_at_once(lib, d, backward):
    """Items are shared out evenly over the CTAs: with more than the two an SM that registers allow, some of equal
    size would run alone at the end.  (Without a GPU the plan is that of 148 SMs.)"""
    ctas = ctypes.c_int()
    assert lib.bl_qk_norm_rope_plan(rows(M=100_000, D=d), backward, ctypes.byref(ctas)) == 1
    assert ctas.value == 2 * 148
    assert lib.bl_qk_norm_rope_plan(rows(D=d), backward, ctypes.byref(ctas)) == 0 and 1 <= ctas.value <= 96


def test_plans_of_rows_that_are_refused(lib):
    plan = lib.bl_qk_norm_rope_plan
    assert plan(None, 0, None) == -1 and plan(rows(D=12), 0, None) == -1 and plan(rows(M=0), 1, None) == -1
    assert plan(rows(v=None), 1, None) == 0


def test_workspace_does_not_grow_with_rows_that_no_sequence_has(lib):
    """A buffer for many tokens with a small batch in it: the parts of dK and dV take the sequences' keys."""
    size = lib.bl_attention_backward_workspace_size
    small = dict(Hq=32, Hkv=4, D=128, ldq=4096, ldk=512, ldv=512, max_q=200, max_k=200, B=2)
    parts = size(call(**small, Tq=0, q=None, Tk=400))
    assert parts > 2 * 8 * 2 * 200 * 4 * 128 * 4
    assert size(call(**small, Tq=0, q=None, Tk=1 << 28)) == parts
    for b, most in ((1, 1 << 28), (147, 128), (3, 6000), (1, 18000)):
        assert size(call(**{**small, "B": b, "max_k": most, "Hkv": 1, "Hq": 32, "ldk": 128, "ldv": 128}, Tq=0, q=None, Tk=1 << 28)) < 40 << 20
