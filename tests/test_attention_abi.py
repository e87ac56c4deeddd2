"""Host-side checks of the attention operators' C ABI: every refusal happens
before any CUDA call, struct layouts match the header, workspace sizes."""
import ctypes
import os
import subprocess

import pytest

import int8_row_absmax_b200 as pkg
from int8_row_absmax_b200 import attn
from int8_row_absmax_b200 import build as blbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, INVALID, ALIGN, WS, OK = None, 1, 2, 4, 0


@pytest.fixture(scope="module")
def lib():
    blbuild.build()
    return pkg.load()


@pytest.mark.parametrize("struct,cls", [("bl_qkv_rows", attn.QkvRows), ("bl_kv_pages", attn.KvPages),
                                        ("bl_attn_call", attn.AttnCall)])
def test_struct_layouts(tmp_path, struct, cls):
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"bitlinear.h\"\nint main(void){\n"
                   f"printf(\"%zu\\n\", sizeof({struct}));\n" +
                   "".join(f"printf(\"%zu\\n\", offsetof({struct}, {f}));\n" for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src), "-o",
                    str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def rows(**kw):
    d = dict(M=2, Hq=4, Hkv=2, D=32, q=16, k=16, v=16, ldq=128, ldk=64, ldv=64, pos=16, table=16, P=10, R=32,
             interleaved=0, gq=16, gk=None, eps=1e-6)
    d.update(kw)
    return ctypes.byref(attn.QkvRows(**d))


def pages(**kw):
    d = dict(t=2, k=16, v=16, pages=8, page=16, Hkv=2, D=32)
    d.update(kw)
    return ctypes.byref(attn.KvPages(**d))


def call(**kw):
    d = dict(t=2, Hq=4, Hkv=2, D=64, q=16, k=16, v=16, ldq=256, ldk=128, ldv=128, Tq=10, Tk=10, cu_q=16, cu_k=16, B=1,
             max_q=10, max_k=10, window=0, sinks=0, scale=0.125)
    d.update(kw)
    return ctypes.byref(attn.AttnCall(**d))


BAD_ROWS = [(dict(M=-1), INVALID), (dict(M=1 << 29), INVALID), (dict(Hq=5), INVALID), (dict(Hkv=0), INVALID), (dict(D=12), INVALID),
            (dict(D=264), INVALID), (dict(R=12), INVALID), (dict(R=40), INVALID), (dict(R=-8), INVALID),
            (dict(interleaved=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
            (dict(P=0), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(pos=None), INVALID),
            (dict(table=None), INVALID), (dict(ldq=124), INVALID), (dict(ldk=60), INVALID), (dict(ldk=66), ALIGN),
            (dict(q=8), ALIGN), (dict(gq=20), ALIGN), (dict(table=24), ALIGN), (dict(pos=18), ALIGN)]


@pytest.mark.parametrize("kw,expect", BAD_ROWS + [(dict(v=None), INVALID), (dict(ldv=60), INVALID)])
def test_norm_rope_refusals(lib, kw, expect):
    assert lib.bl_qk_norm_rope(rows(**kw), 2, 16, 16, 16, NULL) == expect
    assert lib.bl_qk_norm_rope_append(rows(**kw), 16, pages(), 16, NULL) == expect


@pytest.mark.parametrize("kw,expect", BAD_ROWS)
def test_norm_rope_backward_refusals(lib, kw, expect):
    f = lib.bl_qk_norm_rope_backward
    assert f(rows(**kw), 2, 16, 16, 16, 16, 128, 16, 64, 16, 64, 16, 16, 256, 1 << 20, NULL) == expect
    assert lib.bl_qk_norm_rope_backward_workspace_size(rows(**kw)) == 0


def test_norm_rope_more_refusals(lib):
    f, ap, bw = lib.bl_qk_norm_rope, lib.bl_qk_norm_rope_append, lib.bl_qk_norm_rope_backward
    assert f(NULL, 2, 16, 16, 16, NULL) == INVALID
    assert f(rows(), 3, 16, 16, 16, NULL) == INVALID                     # no such type
    assert f(rows(), 2, NULL, 16, 16, NULL) == INVALID
    assert f(rows(), 2, 16, 24, 16, NULL) == ALIGN
    assert f(rows(M=0, q=None, k=None, v=None, pos=None, table=None), 2, NULL, NULL, NULL, NULL) == OK
    for kw, e in ((dict(t=0), INVALID), (dict(k=None), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
                  (dict(Hkv=1), INVALID), (dict(D=64), INVALID), (dict(page=1 << 26), INVALID),
                  (dict(v=24), ALIGN)):
        assert ap(rows(), 16, pages(**kw), 16, NULL) == e
    assert ap(rows(), 16, NULL, 16, NULL) == INVALID
    assert ap(rows(), 16, pages(), NULL, NULL) == INVALID
    assert ap(rows(), 16, pages(), 20, NULL) == ALIGN
    good = [rows(), 2, 16, 16, 16, 16, 128, 16, 64, 16, 64, 16, 16, 256, 1 << 20, NULL]
    for at, value, e in ((1, 7, INVALID), (2, NULL, INVALID), (5, NULL, INVALID), (6, 120, INVALID), (6, 130, ALIGN),
                         (7, 20, ALIGN), (11, 18, ALIGN), (13, NULL, WS), (13, 128, WS), (14, 16, WS)):
        args = list(good)
        args[at] = value
        assert bw(*args) == e, (at, value)
    assert lib.bl_qk_norm_rope_backward_workspace_size(rows()) >= 2 * 32 * 4


def test_rope_table_refusals(lib):
    f = lib.bl_rope_table
    for args in ((NULL, 4, 8, 1e4), (16, 0, 8, 1e4), (16, 4, 7, 1e4), (16, 4, 0, 1e4), (16, 4, 8, 0.0),
                 (16, 4, 8, float("inf")), (16, 1 << 40, 8, 1e4)):
        assert f(*args, NULL) == INVALID
    assert f(18, 4, 8, 1e4, NULL) == ALIGN


BAD_CALLS = [(dict(t=0), INVALID), (dict(Hq=3), INVALID), (dict(D=60), INVALID), (dict(D=136), INVALID),
             (dict(Tq=-1), INVALID), (dict(Tk=1 << 29), INVALID), (dict(B=-1), INVALID), (dict(window=-1), INVALID),
             (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
             (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID),
             (dict(ldq=248), INVALID), (dict(ldv=120), INVALID), (dict(ldq=260), ALIGN), (dict(k=24), ALIGN),
             (dict(cu_q=18), ALIGN), (dict(max_q=-1), INVALID)]


@pytest.mark.parametrize("kw,expect", BAD_CALLS)
def test_attention_refusals(lib, kw, expect):
    assert lib.bl_attention(call(**kw), 16, 16, NULL) == expect
    assert lib.bl_attention_backward(call(**kw), 16, 16, 16, 16, 16, 16, 256, 1 << 30, NULL) == expect
    assert lib.bl_attention_backward_workspace_size(call(**kw)) == 0


def test_attention_more_refusals(lib):
    f, bw = lib.bl_attention, lib.bl_attention_backward
    assert f(NULL, 16, 16, NULL) == INVALID
    assert f(call(), NULL, 16, NULL) == INVALID
    assert f(call(), 24, 16, NULL) == ALIGN
    assert f(call(B=0, q=None, cu_q=None, cu_k=None), NULL, NULL, NULL) == OK
    assert f(call(Tq=0, q=None), NULL, NULL, NULL) == OK
    good = [call(), 16, 16, 16, 16, 16, 16, 256, 1 << 30, NULL]
    for at in (1, 2, 3, 4, 5, 6):
        args = list(good)
        args[at] = NULL
        assert bw(*args) == INVALID
        args[at] = 17
        assert bw(*args) == ALIGN
    for at, value in ((7, NULL), (7, 128), (8, 16)):
        args = list(good)
        args[at] = value
        assert bw(*args) == WS
    assert lib.bl_attention_backward_workspace_size(call()) >= 10 * 4 * 4


def test_paged_attention_refusals(lib):
    f = lib.bl_paged_attention
    good = dict(q=16, B=2, Hq=4, c=pages(), table=16, ldt=4, lens=16, window=0, sinks=0, scale=0.2, out_t=0, out=16,
                ws=256, n=1 << 30, st=NULL)

    def run(**kw):
        d = dict(good)
        d.update(kw)
        return f(*d.values())
    for kw, e in ((dict(c=NULL), INVALID), (dict(c=pages(t=0)), INVALID), (dict(c=pages(D=136)), INVALID),
                  (dict(c=pages(k=24)), ALIGN), (dict(B=-1), INVALID), (dict(Hq=3), INVALID), (dict(ldt=0), INVALID),
                  (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=-1.0), INVALID),
                  (dict(out_t=1), INVALID), (dict(q=NULL), INVALID), (dict(table=NULL), INVALID),
                  (dict(lens=NULL), INVALID), (dict(out=NULL), INVALID), (dict(q=24), ALIGN), (dict(lens=18), ALIGN),
                  (dict(ws=NULL), WS), (dict(ws=128), WS), (dict(n=64), WS), (dict(B=0, q=NULL, ws=NULL), OK)):
        assert run(**kw) == e, kw
    assert lib.bl_paged_attention_workspace_size(2, 4, pages()) % 256 == 0
    assert lib.bl_paged_attention_workspace_size(2, 3, pages()) == 0
