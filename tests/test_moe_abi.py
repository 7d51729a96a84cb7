"""include/rd_moe.h on the host: it compiles as C, every symbol is exported, bad arguments are
rejected before any CUDA call."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rd_moe.h")
OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
P = 0x100000          # fake device addresses far apart: never dereferenced on these paths


def addr(i):
    return P + (i << 40)


class Config(ctypes.Structure):
    _fields_ = [("topk", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


@pytest.fixture(scope="module")
def lib():
    from expert_ffn_ragged_gb300 import build, moe

    lib = ctypes.CDLL(build.build())
    moe.declare(lib)
    lib.rd_mxfp4_scale_width.argtypes = [ctypes.c_int64]
    lib.rd_mxfp4_scale_width.restype = ctypes.c_int64
    return lib


def test_header_symbols_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(rd_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted([
        "rd_route", "rd_route_bwd", "rd_sort_rows", "rd_dispatch_rows", "rd_combine_rows",
        "rd_combine_rows_bwd", "rd_mxfp4_scale_width", "rd_mxfp4_quantize",
        "rd_mxfp4_quantize_weights", "rd_mxfp4_dequantize", "rd_ragged_dot_mxfp4"])
    out = subprocess.run(["nm", "-D", "--defined-only", lib._name], capture_output=True, text=True)
    exported = set(re.findall(r"\bT (rd_[a-z0-9_]+)\b", out.stdout))
    assert set(declared) <= exported


def test_header_compiles_as_c(tmp_path):
    cc = shutil.which("cc") or shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "rd_moe.h"\nint main(void) { rd_route_config c = {1, RD_SCORE_SIGMOID, 1, 1, 0, 1.0f};'
                   ' return (int)rd_mxfp4_scale_width(c.topk); }\n')
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-c", str(src), "-I", os.path.join(ROOT, "include"),
                    "-o", str(tmp_path / "t.o")], check=True)


def test_scale_width(lib):
    import expert_ffn_ragged_gb300 as rd

    for k, want in ((0, 0), (32, 16), (512, 16), (544, 32), (4096, 128), (768, 32)):
        assert lib.rd_mxfp4_scale_width(k) == want == rd.mxfp4_scale_width(k)


def test_route_refusals(lib):
    ok = dict(logits=addr(1), dtype=0, bias=addr(2), tokens=4, experts=16, limit=None, ids=addr(3),
              weights=addr(4), sizes=addr(5), pos=addr(6), rows=addr(7))
    good = dict(topk=2, score=0, groups=4, topk_groups=2, renormalize=1, scale=1.0)

    def call(cfg=None, null=False, **kw):
        a = dict(ok, **kw)
        c = Config(**dict(good, **(cfg or {})))
        return lib.rd_route(a["logits"], a["dtype"], a["bias"], a["tokens"], a["experts"],
                            None if null else ctypes.byref(c), a["limit"], a["ids"], a["weights"],
                            a["sizes"], a["pos"], a["rows"], None)

    assert call(null=True) == INVALID
    for kw in (dict(tokens=-1), dict(experts=0), dict(dtype=2), dict(logits=None), dict(ids=None),
               dict(weights=None), dict(sizes=None), dict(pos=None), dict(rows=None),
               dict(ids=ok["logits"]), dict(pos=ok["ids"]), dict(weights=ok["bias"]),
               dict(limit=ok["rows"])):
        assert call(**kw) == INVALID, kw
    for cfg in (dict(topk=0), dict(topk=17), dict(score=2), dict(groups=0), dict(groups=3),
                dict(topk_groups=0), dict(topk_groups=5), dict(renormalize=2)):
        assert call(cfg) == INVALID, cfg
    assert call(experts=2048, cfg=dict(groups=1, topk_groups=1)) == UNSUPPORTED
    assert call(experts=64, cfg=dict(topk=33, groups=1, topk_groups=1)) == UNSUPPORTED
    assert call(experts=128, cfg=dict(groups=64)) == UNSUPPORTED
    assert call(tokens=1 << 40) == UNSUPPORTED
    assert call(logits=ok["logits"] + 2) == UNSUPPORTED      # an f32 row off its 4 bytes
    assert call(ids=ok["ids"] + 1) == UNSUPPORTED
    assert call(limit=addr(8) + 2) == UNSUPPORTED


def test_route_bwd_and_sort_refusals(lib):
    c = Config(2, 0, 1, 1, 1, 1.0)

    def bwd(logits=addr(1), dtype=0, ids=addr(2), d=addr(3), out=addr(4), tokens=4, experts=16, cfg=c):
        return lib.rd_route_bwd(logits, dtype, ids, d, tokens, experts,
                                None if cfg is None else ctypes.byref(cfg), None, out, None)

    for kw in (dict(cfg=None), dict(logits=None), dict(ids=None), dict(d=None), dict(out=None),
               dict(out=addr(1)), dict(out=addr(3)), dict(dtype=7), dict(tokens=-2)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(out=addr(4) + 2) == UNSUPPORTED

    def sort(ids=addr(1), tokens=4, topk=2, experts=8, sizes=addr(2), pos=addr(3), rows=addr(4)):
        return lib.rd_sort_rows(ids, tokens, topk, experts, None, sizes, pos, rows, None)

    for kw in (dict(ids=None), dict(sizes=None), dict(pos=None), dict(rows=None), dict(tokens=-1),
               dict(topk=0), dict(experts=0), dict(pos=addr(1)), dict(rows=addr(2))):
        assert sort(**kw) == INVALID, kw
    assert sort(experts=1025) == UNSUPPORTED
    assert sort(tokens=1 << 30, topk=4) == UNSUPPORTED
    assert sort(pos=addr(3) + 2) == UNSUPPORTED


def test_row_mover_refusals(lib):
    def dispatch(x=addr(1), pos=addr(2), out=addr(3), t=4, k=2, h=64, rows=8, limit=None):
        return lib.rd_dispatch_rows(x, pos, out, t, k, h, rows, limit, None)

    for kw in (dict(x=None), dict(pos=None), dict(out=None), dict(out=addr(1)), dict(t=-1), dict(k=0),
               dict(h=-8), dict(rows=-1)):
        assert dispatch(**kw) == INVALID, kw
    for kw in (dict(h=12), dict(k=33), dict(x=addr(1) + 8), dict(out=addr(3) + 2), dict(limit=addr(5) + 1),
               dict(t=1 << 33)):
        assert dispatch(**kw) == UNSUPPORTED, kw

    def combine(y=addr(1), pos=addr(2), w=addr(3), out=addr(4), t=4, k=2, h=64, rows=8):
        return lib.rd_combine_rows(y, pos, w, out, t, k, h, rows, None, None)

    for kw in (dict(y=None), dict(pos=None), dict(out=None), dict(out=addr(1)), dict(out=addr(3))):
        assert combine(**kw) == INVALID, kw
    assert combine(w=addr(3) + 1) == UNSUPPORTED

    def bwd(d=addr(1), y=addr(2), pos=addr(3), w=addr(4), dy=addr(5), dw=addr(6), t=4, k=2, h=64, rows=8):
        return lib.rd_combine_rows_bwd(d, y, pos, w, dy, dw, t, k, h, rows, None, None)

    for kw in (dict(d=None), dict(y=None), dict(pos=None), dict(w=None), dict(dy=None), dict(dw=None),
               dict(dy=addr(2)), dict(dw=addr(4)), dict(dw=addr(5))):
        assert bwd(**kw) == INVALID, kw
    assert bwd(dw=addr(6) + 2) == UNSUPPORTED


def test_mxfp4_refusals(lib):
    def quant(x=addr(1), pos=None, q=addr(2), s=addr(3), rows=4, topk=1, k=64, out=4):
        return lib.rd_mxfp4_quantize(x, pos, q, s, rows, topk, k, out, None, None)

    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(rows=-1), dict(out=3), dict(q=addr(1)),
               dict(s=addr(2)), dict(pos=addr(4), topk=0)):
        assert quant(**kw) == INVALID, kw
    for kw in (dict(k=48), dict(q=addr(2) + 8), dict(pos=addr(4), topk=33), dict(pos=addr(4) + 1)):
        assert quant(**kw) == UNSUPPORTED, kw

    def weights(rhs=addr(1), q=addr(2), s=addr(3), g=2, k=64, n=64):
        return lib.rd_mxfp4_quantize_weights(rhs, q, s, g, k, n, None)

    for kw in (dict(rhs=None), dict(q=None), dict(s=None), dict(g=-1), dict(s=addr(1))):
        assert weights(**kw) == INVALID, kw
    for kw in (dict(k=40), dict(n=12), dict(g=70000), dict(k=1 << 22), dict(rhs=addr(1) + 2)):
        assert weights(**kw) == UNSUPPORTED, kw
    assert lib.rd_mxfp4_dequantize(addr(1), addr(2), addr(1), 4, 64, None, None) == INVALID
    assert lib.rd_mxfp4_dequantize(addr(1), addr(2), addr(3), 4, 40, None, None) == UNSUPPORTED

    def dot(a=addr(1), a_s=addr(2), b=addr(3), b_s=addr(4), out=addr(5), out_s=None, m=16, k=64, n=64,
            gs=addr(7), gt=4, off=0, gl=4, limit=None, epi=0, status=None):
        return lib.rd_ragged_dot_mxfp4(a, a_s, b, b_s, out, out_s, m, k, n, gs, gt, off, gl, limit, epi,
                                       status, None)

    for kw in (dict(a=None), dict(a_s=None), dict(b=None), dict(b_s=None), dict(out=None), dict(gs=None),
               dict(epi=3), dict(epi=2), dict(out_s=addr(6)), dict(off=2, gl=3), dict(gl=0), dict(m=-1),
               dict(out=addr(1)), dict(out=addr(4)), dict(epi=2, out_s=addr(2)), dict(epi=2, out_s=addr(5)),
               dict(status=addr(5))):
        assert dot(**kw) == INVALID, kw
    for kw in (dict(k=40), dict(n=12), dict(epi=1, n=40), dict(epi=2, n=96, out_s=addr(6)),
               dict(a=addr(1) + 8), dict(b_s=addr(4) + 4), dict(gt=2000)):
        assert dot(**kw) == UNSUPPORTED, kw


def test_binding_refuses_before_the_library():
    import torch

    import expert_ffn_ragged_gb300 as rd

    cpu = torch.zeros(2, 8)
    ids = torch.zeros(2, 2, dtype=torch.int32)
    rows = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: rd.route(cpu, 2), lambda: rd.route(cpu.half(), 2),
                 lambda: rd.route_bwd(cpu, ids, torch.zeros(2, 2)), lambda: rd.sort_rows(ids, 4),
                 lambda: rd.dispatch_rows(rows, ids), lambda: rd.combine_rows(rows, ids),
                 lambda: rd.combine_rows_bwd(rows, rows, ids, torch.zeros(2, 2)),
                 lambda: rd.mxfp4_quantize(rows), lambda: rd.mxfp4_quantize_weights(rows[None]),
                 lambda: rd.mxfp4_dequantize(torch.zeros(1, 16, dtype=torch.uint8), None),
                 lambda: rd.ragged_dot_mxfp4(torch.zeros(1, 16, dtype=torch.uint8), None, None, None, None)):
        with pytest.raises(ValueError):
            call()
