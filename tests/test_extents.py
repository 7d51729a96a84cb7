"""Extents near 2^31: the schedule's counts stay right, and what a call cannot index is refused before any
CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "expert_ffn_ragged_gb300", "csrc")
FWD, DX, DW = 0, 1, 2
TOP = 2 ** 31
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("extent") / "libextent.so")
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC,
                    os.path.join(HERE, "extent_probe.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.group_tiles.restype = ctypes.c_longlong
    return lib


@pytest.mark.parametrize("rows", [1, 128, 129, TOP - 512, TOP - 256, TOP - 255, TOP - 129, TOP - 128, TOP - 2, TOP - 1])
@pytest.mark.parametrize("first", [0, 1])
def test_rows_of_one_group(probe, rows, first):
    if first + rows > TOP - 1:
        pytest.skip("past the largest m")
    end = first + rows
    for tm in (32, 128, 256):
        assert probe.group_tiles(FWD, first, end, tm, 3) == 3 * -(-rows // tm)
    out = (ctypes.c_int32 * 4)()
    for tm in (128, 256):
        tiles = -(-rows // tm)
        for t in {0, tiles // 2, tiles - 1}:
            probe.decode_tile_of(0, tm, first, end, 64, t, out)
            assert list(out)[:3] == [t, end - tm if t == tiles - 1 else first + t * tm, 1]
    probe.decode_tile_of(1, 128, first, end, 0, 0, out)
    assert out[2] == -(-rows // 64) and out[3] == end - 64


@pytest.mark.parametrize("kc", [8, 64, 72, TOP - 128, TOP - 64, TOP - 56, TOP - 8])
def test_contraction_length(probe, kc):
    out = (ctypes.c_int32 * 4)()
    probe.decode_tile_of(0, 128, 0, 100, kc, 0, out)
    assert out[2] == -(-kc // 64)


@pytest.fixture(scope="module")
def lib():
    import expert_ffn_ragged_gb300 as rd
    from expert_ffn_ragged_gb300 import build

    build.build()
    return rd.load()


def _at(i):
    return (i + 1) << 44          # addresses far apart, never dereferenced


def test_widths_that_no_tile_can_index(lib):
    """Output widths above 2^31 - 256, and of the 4-bit product a k above 2^31 - 1024."""
    gs = _at(9)

    def fwd(n, epi=0):
        return lib.rd_ragged_dot(_at(0), _at(1), _at(2), 1, 8, n, gs, 1, 0, 1, None, epi, None, None)

    def dx(k):
        return lib.rd_ragged_dot_trans_rhs(_at(0), _at(1), _at(2), 1, k, 8, gs, 1, 0, 1, None, None, None)

    def dx_glu(f):
        return lib.rd_ragged_dot_trans_rhs_glu_bwd(_at(0), _at(1), _at(3), _at(2), 1, f, 8, gs, 1, 0, 1, None, None, None)

    def dw(k, n):
        return lib.rd_trans_ragged_dot(_at(0), _at(1), _at(2), 1, k, n, gs, 1, 0, 1, None, None, 0, None, None)

    def dw_plain(k, n):
        return lib.rd_trans_ragged_dot_no_alloc(_at(0), _at(1), _at(2), 1, k, n, gs, 1, 0, 1, None, None, None)

    def dw_f32(k, n):
        return lib.rd_trans_ragged_dot_f32(_at(0), _at(1), _at(2), 1, k, n, gs, 1, 0, 1, None, 0, None, 0, None, None)

    def four(k, n):
        return lib.rd_ragged_dot_mxfp4(_at(0), _at(1), _at(2), _at(3), _at(4), None, 1, k, n, gs, 1, 0, 1, None, 0, None,
                                       None)

    top, fits = TOP - 8, TOP - 256
    codes = [fwd(top), dx(top), dx_glu(top), dw(top, 8), dw(8, top), dw_plain(top, 8), dw_f32(top, 8), dw_f32(8, top),
             four(32, top), four(TOP - 32, 8), four(TOP - 992, 8), fwd(fits + 8), dx(fits + 8), dw(fits + 8, 8),
             dw(8, fits + 8), four(32, fits + 8)]
    assert codes == [UNSUPPORTED] * len(codes)
    if not _gpu():
        # accepted as far as the machine without a GPU goes: past the checks, refused by the device's
        codes = [fwd(fits), fwd(TOP - 16, 1), dx(fits), dw(fits, 8), dw(8, fits), four(32, fits), four(TOP - 1024, 8)]
        assert not {0, 1, UNSUPPORTED} & set(codes)


def _gpu():
    import torch

    return torch.cuda.is_available()
