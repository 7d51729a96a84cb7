"""include/rd_block.h on the host: it compiles as C, every symbol is exported, bad arguments are
rejected before any CUDA call."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rd_block.h")
OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
NAN, INF = float("nan"), float("inf")


def addr(i):
    return 0x100000 + (i << 40)       # fake device addresses far apart: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from expert_ffn_ragged_gb300 import block, build

    lib = ctypes.CDLL(build.build())
    block.declare(lib)
    return lib


def test_header_symbols_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(rd_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted([
        "rd_layer_norm_fwd", "rd_layer_norm_bwd", "rd_layer_norm_bwd_workspace_size", "rd_linear",
        "rd_linear_act_bwd", "rd_linear_act_bwd_workspace_size", "rd_dropout_rows"])
    out = subprocess.run(["nm", "-D", "--defined-only", lib._name], capture_output=True, text=True)
    assert set(declared) <= set(re.findall(r"\bT (rd_[a-z0-9_]+)\b", out.stdout))


def test_header_compiles_as_c(tmp_path):
    cc = shutil.which("cc") or shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "rd_block.h"\nint main(void) { size_t n = 0;'
                   ' return (int)rd_linear_act_bwd_workspace_size(4, 8, RD_ACT_RELU, &n); }\n')
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-c", str(src), "-I", os.path.join(ROOT, "include"),
                    "-o", str(tmp_path / "t.o")], check=True)


def _refused(call, invalid, unsupported):
    for kw in invalid:
        assert call(**kw) == INVALID, kw
    for kw in unsupported:
        assert call(**kw) == UNSUPPORTED, kw
    assert call() in (OK, CUDA, UNSUPPORTED) and call() != INVALID      # past the checks, without a GPU here


def test_norm_refusals(lib):
    def fwd(x=addr(1), dtype=0, w=addr(2), b=addr(3), eps=1e-5, out=addr(4), out_dtype=1, mean=addr(5), rstd=addr(6),
            rows=4, hidden=64, limit=addr(7)):
        return lib.rd_layer_norm_fwd(x, dtype, w, b, eps, out, out_dtype, mean, rstd, rows, hidden, limit, None)

    if lib.rd_layer_norm_fwd(None, 0, None, None, 1.0, None, 0, None, None, 0, 8, None, None) == OK:
        pytest.skip("a GPU is there: the fake addresses would be launched on")
    _refused(fwd,
             [dict(x=None), dict(out=None), dict(mean=None), dict(rstd=None), dict(dtype=2), dict(out_dtype=-1),
              dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(rows=-1), dict(hidden=-8), dict(out=addr(1)),
              dict(mean=addr(2)), dict(rstd=addr(5)), dict(out=addr(1) + 512), dict(limit=addr(6))],
             [dict(hidden=12), dict(rows=1 << 31), dict(hidden=1 << 31), dict(x=addr(1) + 16), dict(out=addr(4) + 8),
              dict(w=addr(2) + 4), dict(b=addr(3) + 8), dict(mean=addr(5) + 2), dict(limit=addr(7) + 1)])

    def bwd(d=addr(1), out_dtype=1, x=addr(2), dtype=0, w=addr(3), mean=addr(4), rstd=addr(5), d_x=addr(6),
            dw=addr(7), db=addr(8), rows=1 << 20, hidden=64, limit=None, ws=addr(9), nb=1 << 30):
        return lib.rd_layer_norm_bwd(d, out_dtype, x, dtype, w, mean, rstd, d_x, dw, db, rows, hidden, limit, ws, nb, None)

    _refused(bwd,
             [dict(d=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(d_x=None), dict(ws=None),
              dict(d_x=addr(2)), dict(d_x=addr(1)), dict(dw=addr(8)), dict(ws=addr(6)), dict(db=addr(3)),
              dict(dtype=9), dict(rows=-1), dict(ws=addr(4))],
             [dict(hidden=4), dict(ws=addr(9) + 16), dict(d_x=addr(6) + 16), dict(d=addr(1) + 8), dict(rstd=addr(5) + 1),
              dict(dw=addr(7) + 4)])
    size = ctypes.c_size_t(0)
    assert lib.rd_layer_norm_bwd_workspace_size(4, 64, None) == INVALID
    assert lib.rd_layer_norm_bwd_workspace_size(-4, 64, ctypes.byref(size)) == INVALID
    assert lib.rd_layer_norm_bwd_workspace_size(4, 63, ctypes.byref(size)) == UNSUPPORTED


def test_linear_refusals(lib):
    def lin(x=addr(1), w=addr(2), b=addr(3), res=addr(4), act=2, out=addr(5), out_dtype=1, pre=addr(6), m=4, k=64,
            n=64, gs=None, g=1, off=0, gl=1, limit=None, status=addr(8)):
        return lib.rd_linear(x, w, b, res, act, out, out_dtype, pre, m, k, n, gs, g, off, gl, limit, status, None)

    if lin(m=0) == OK:
        pytest.skip("a GPU is there: the fake addresses would be launched on")
    _refused(lin,
             [dict(x=None), dict(w=None), dict(out=None), dict(act=5), dict(act=-1), dict(out_dtype=2), dict(m=-1),
              dict(k=-8), dict(n=-8), dict(g=2), dict(gl=2), dict(off=1), dict(gs=addr(9), g=0), dict(gs=addr(9), g=2, off=1, gl=2),
              dict(out=addr(1)), dict(out=addr(2)), dict(out=addr(4)), dict(pre=addr(5)), dict(pre=addr(1)),
              dict(out=addr(3)), dict(limit=addr(5)), dict(status=addr(6))],
             [dict(k=12), dict(n=12), dict(m=1 << 31), dict(n=(1 << 31) - 248), dict(gs=addr(9), g=1025, gl=1025),
              dict(x=addr(1) + 8), dict(w=addr(2) + 2), dict(out_dtype=0, out=addr(5) + 16),
              dict(out_dtype=0, res=addr(4) + 16), dict(pre=addr(6) + 8), dict(b=addr(3) + 4),
              dict(gs=addr(9) + 2), dict(limit=addr(7) + 1)])

    def bwd(d=addr(1), out_dtype=1, pre=addr(2), act=4, d_pre=addr(3), d_bias=addr(4), m=1100, n=64, gs=None, g=1, off=0,
            gl=1, limit=None, ws=addr(5), nb=1 << 20, status=None):
        return lib.rd_linear_act_bwd(d, out_dtype, pre, act, d_pre, d_bias, m, n, gs, g, off, gl, limit, ws, nb, status, None)

    _refused(bwd,
             [dict(d=None), dict(pre=None), dict(act=0), dict(act=7), dict(out_dtype=3), dict(ws=None), dict(nb=64),
              dict(d_pre=addr(1)), dict(d_pre=addr(2)), dict(d_bias=addr(3)), dict(ws=addr(2)), dict(ws=addr(4)),
              dict(m=-1), dict(g=3), dict(gs=addr(6), g=4, off=3, gl=2), dict(limit=addr(4))],
             [dict(n=12), dict(m=1 << 31), dict(gs=addr(6), g=2000, gl=2000), dict(ws=addr(5) + 16),
              dict(d_bias=addr(4) + 4), dict(out_dtype=0, d=addr(1) + 16), dict(d_pre=addr(3) + 2)])
    size = ctypes.c_size_t(0)
    assert lib.rd_linear_act_bwd_workspace_size(4, 64, 1, None) == INVALID
    assert lib.rd_linear_act_bwd_workspace_size(4, 64, 0, ctypes.byref(size)) == INVALID
    assert lib.rd_linear_act_bwd_workspace_size(4, 64, 2000, ctypes.byref(size)) == UNSUPPORTED
    assert lib.rd_linear_act_bwd_workspace_size(3000, 64, 3, ctypes.byref(size)) == OK
    assert size.value >= 4 * 64 * (3000 // 64 + 3)
    assert lib.rd_linear_act_bwd_workspace_size(4, 64, 1, ctypes.byref(size)) == OK and size.value == 0


def test_dropout_refusals(lib):
    def drop(x=addr(1), dtype=1, res=addr(2), rng=addr(3), p=0.1, out=addr(4), out_dtype=0, rows=4, hidden=64, limit=None):
        return lib.rd_dropout_rows(x, dtype, res, rng, p, out, out_dtype, rows, hidden, limit, None)

    if drop(rows=0) == OK:
        pytest.skip("a GPU is there: the fake addresses would be launched on")
    _refused(drop,
             [dict(x=None), dict(out=None), dict(rng=None), dict(p=-0.1), dict(p=1.5), dict(p=NAN), dict(dtype=2),
              dict(out_dtype=2), dict(rows=-1), dict(out=addr(1)), dict(out=addr(2)), dict(rng=addr(4)), dict(limit=addr(4))],
             [dict(hidden=20), dict(rows=1 << 31), dict(x=addr(1) + 8), dict(out=addr(4) + 16), dict(res=addr(2) + 16),
              dict(rng=addr(3) + 4), dict(limit=addr(5) + 2)])
